"""Gradients of the expert-grouped products (tkg_gemm_grouped_dev_bf16_dgrad,
_wgrad) against their formulas in 64 bits and, the products being bilinear,
against differences: ragged and empty groups, counts that overrun the capacity,
rows outside the groups that hold anything, both output types.

Tolerances: the library's acceptance bound for its products, 2^-7 |ref| + 1e-5
sum |a b| (BF16 results); for FP32 results 1e-5 sum |a b| plus one FP32 rounding
of what is stored."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
GUARD = 7.0


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK
    tkg.set_option(tkg.OPT_BF16_TILE_N, 0)


def cut(sizes, cap):
    """First row and rows of each group: negative counts are 0, rows past the capacity are cut off."""
    out, row = [], 0
    for m in sizes:
        m = min(max(m, 0), cap - row)
        out.append((row, m))
        row += m
    return out, row


class Groups:
    def __init__(self, sizes, n, k, spare=0, seed=0, alpha=1.0, fill=float("nan"), cap=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed * 131 + n * 7 + k + len(sizes))
        self.sizes, self.n, self.k, self.alpha = list(sizes), n, k, alpha
        self.cap = sum(max(s, 0) for s in sizes) + spare if cap is None else cap
        self.spans, self.rows = cut(sizes, self.cap)
        self.dev = torch.tensor(sizes, dtype=torch.int32, device="cuda")
        r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
        self.dD, self.A, self.B = r(self.cap, n), r(self.cap, k), r(len(sizes), n, k)
        for t in (self.dD, self.A):
            t[self.rows:] = fill

    def dgrad(self):
        ref = torch.zeros(self.rows, self.k, device="cuda", dtype=F64)
        mag = torch.zeros_like(ref)
        for g, (o, m) in enumerate(self.spans):
            d, b = self.dD[o:o + m].to(F64), self.B[g].to(F64)
            ref[o:o + m], mag[o:o + m] = self.alpha * (d @ b), abs(self.alpha) * (d.abs() @ b.abs())
        return ref, mag

    def wgrad(self):
        refs, mags = [], []
        for o, m in self.spans:
            d, a = self.dD[o:o + m].to(F64), self.A[o:o + m].to(F64)
            refs.append(self.alpha * (d.T @ a))
            mags.append(abs(self.alpha) * (d.abs().T @ a.abs()))
        return torch.stack(refs), torch.stack(mags)


def within(got, ref, bound, what):
    err = (got.to(F64) - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside tolerance"


def check_dgrad(p):
    dA = torch.full((p.cap, p.k), GUARD, device="cuda", dtype=BF16)
    tkg.gemm_grouped_dev_bf16_dgrad(p.dev, p.dD, p.B, dA, alpha=p.alpha)
    ref, mag = p.dgrad()
    within(dA[:p.rows], ref, 2.0 ** -7 * ref.abs() + 1e-5 * mag, f"dgrad {p.sizes} n={p.n} k={p.k}")
    assert (dA[p.rows:] == GUARD).all(), "rows outside the groups were written"
    return dA


def check_wgrad(p, dtype=BF16):
    dB = torch.full((len(p.sizes), p.n, p.k), GUARD, device="cuda", dtype=dtype)
    tkg.gemm_grouped_dev_bf16_wgrad(p.dev, p.dD, p.A, dB, alpha=p.alpha)
    ref, mag = p.wgrad()
    bound = 1e-5 * mag + (2.0 ** -7 if dtype == BF16 else 2.0 ** -23) * ref.abs()
    within(dB, ref, bound, f"wgrad {p.sizes} n={p.n} k={p.k}")
    return dB


SIZES = [
    [128, 256, 384], [1, 0, 300, 129, 7], [0, 0, 5], [500], [1], [2, 1, 1], [16] * 8, [15, 17, 33, 63, 64, 65],
    [255, 257, 0, 31, 1000], [0, 1, 0],
]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("n,k", [(264, 520), (64, 8), (8, 64), (1000, 256), (136, 2056)])
def test_both_gradients_match_formulas(sizes, n, k):
    p = Groups(sizes, n, k, spare=3, alpha=0.5)
    check_dgrad(p)
    check_wgrad(p)


@pytest.mark.parametrize("tile_n", [256, 512])
@pytest.mark.parametrize("sizes,n,k", [([3, 200, 0, 129, 40], 264, 520), ([5, 6], 72, 80), ([700, 65, 1, 0], 1000, 1288),
                                       ([640], 512, 768), ([31, 33], 8, 2056)])
def test_wgrad_both_tile_widths(sizes, n, k, tile_n):
    tkg.set_option(tkg.OPT_BF16_TILE_N, tile_n)
    p = Groups(sizes, n, k, spare=70)
    check_wgrad(p)
    g = check_wgrad(p, F32)
    acc = torch.ones_like(g)
    tkg.gemm_grouped_dev_bf16_wgrad(p.dev, p.dD, p.A, acc, accumulate=True)
    for i, (_, m) in enumerate(p.spans):
        assert torch.equal(acc[i], 1 + g[i] if m else torch.ones_like(g[i]))


@pytest.mark.parametrize("sizes", [[40, 0, 300], [1, 2, 3], [0, 0]])
def test_f32_and_accumulation(sizes):
    p = Groups(sizes, 136, 264, spare=9, seed=2)
    g = check_wgrad(p, F32)
    acc = torch.randn_like(g)
    before = acc.clone()
    tkg.gemm_grouped_dev_bf16_wgrad(p.dev, p.dD, p.A, acc, accumulate=True)
    for i, (_, m) in enumerate(p.spans):   # one FP32 addition; groups without rows keep their bits
        assert torch.equal(acc[i], before[i] + g[i] if m else before[i])


def test_many_groups():
    gen = torch.Generator().manual_seed(3)
    sizes = torch.randint(0, 40, (128,), generator=gen).tolist()
    p = Groups(sizes, 72, 136, spare=1)
    check_dgrad(p)
    check_wgrad(p)


@pytest.mark.parametrize("cap", [0, 1, 100, 129, 300])
def test_counts_past_the_capacity_are_cut_off(cap):
    p = Groups([-5, 100, 2 ** 31 - 1, 60, 2 ** 31 - 1], 72, 64, cap=cap)
    if cap == 0:
        dB = torch.full((5, 72, 64), GUARD, device="cuda", dtype=BF16)
        tkg.gemm_grouped_dev_bf16_wgrad(p.dev, p.dD, p.A, dB)
        tkg.gemm_grouped_dev_bf16_dgrad(p.dev, p.dD, p.B, p.A)
        assert (dB == 0).all()
        return
    check_dgrad(p)
    check_wgrad(p)


@pytest.mark.parametrize("fill", [float("inf"), torch.finfo(BF16).min])
def test_rows_outside_the_groups_may_hold_anything(fill):
    p = Groups([30, 0, 77], 264, 136, spare=200, fill=fill)
    check_dgrad(p)
    check_wgrad(p)


def test_an_expert_without_rows_may_hold_anything():
    # n is not a multiple of the 64-row stage: the rows after one expert's last belong to the next one
    p = Groups([40, 0, 30], 72, 136)
    p.B[1] = float("nan")
    check_dgrad(p)


def test_a_row_that_is_not_a_number_stays_in_its_group():
    p = Groups([40, 30, 20], 72, 136, seed=4)
    clean_dA, clean_dB = check_dgrad(p), check_wgrad(p)
    p.dD[45] = float("nan")   # in the second group
    dA, dB = torch.empty_like(clean_dA), torch.empty_like(clean_dB)
    tkg.gemm_grouped_dev_bf16_dgrad(p.dev, p.dD, p.B, dA, alpha=p.alpha)
    tkg.gemm_grouped_dev_bf16_wgrad(p.dev, p.dD, p.A, dB, alpha=p.alpha)
    other = torch.arange(90, device="cuda") != 45
    assert torch.equal(dA[other], clean_dA[other]) and torch.isnan(dA[45]).all()
    assert torch.equal(dB[0], clean_dB[0]) and torch.equal(dB[2], clean_dB[2]) and torch.isnan(dB[1]).all()


def test_one_group_is_the_plain_product():
    p = Groups([777], 512, 768)
    assert torch.equal(check_dgrad(p), check_dgrad(p))
    assert torch.equal(check_wgrad(p), check_wgrad(p))


def test_differences():
    # f = sum(U * D) is linear in A and in B: its central differences are exact up to 64-bit rounding
    p = Groups([33, 0, 70, 5], 136, 72, seed=6)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)

    def f(A, B):
        out = 0.0
        for g, (o, m) in enumerate(p.spans):
            out += float((p.dD[o:o + m].to(F64) * (A[o:o + m] @ B[g].T)).sum())
        return out

    A, B = p.A.to(F64), p.B.to(F64)
    dA, dB = check_dgrad(p), check_wgrad(p)
    (rA, mA), (rB, mB) = p.dgrad(), p.wgrad()
    sA = torch.randn(A.shape, generator=gen, device="cuda", dtype=F64)
    sB = torch.randn(B.shape, generator=gen, device="cuda", dtype=F64)
    for got, ref, mag, step, diff in ((dA, rA, mA, sA, (f(A + sA, B) - f(A - sA, B)) / 2),
                                      (dB, rB, mB, sB, (f(A, B + sB) - f(A, B - sB)) / 2)):
        bound = ((2.0 ** -7 * ref.abs() + 1e-5 * mag) * step.abs()).sum() + 1e-6
        assert abs(float((got.to(F64) * step).sum()) - diff) <= float(bound)


def test_sizes_written_on_the_stream_and_other_stream():
    # the counts come from work queued just before, on a stream of its own, with no host synchronisation
    p = Groups([60, 3, 100], 264, 136, spare=50)
    ref_dA, ref_dB = check_dgrad(p), check_wgrad(p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dev = torch.zeros(3, dtype=torch.int32, device="cuda")
    dA, dB = torch.full_like(ref_dA, GUARD), torch.full_like(ref_dB, GUARD)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            dev.zero_()
            torch.cuda._sleep(2_000_000)
            dev.copy_(p.dev)
        tkg.gemm_grouped_dev_bf16_dgrad(dev, p.dD, p.B, dA, alpha=p.alpha, stream=s)
        tkg.gemm_grouped_dev_bf16_wgrad(dev, p.dD, p.A, dB, alpha=p.alpha, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(dA, ref_dA) and torch.equal(dB, ref_dB)


def test_back_to_back():
    # each call's counts are its own
    ps = [Groups(s, 72, 136, spare=20, seed=i) for i, s in enumerate([[10, 90, 0], [0, 1, 64], [33, 33, 33]])]
    want = [(check_dgrad(p), check_wgrad(p)) for p in ps]
    outs = [(torch.full_like(a, GUARD), torch.full_like(b, GUARD)) for a, b in want]
    for _ in range(5):
        for p, (dA, dB) in zip(ps, outs):
            tkg.gemm_grouped_dev_bf16_dgrad(p.dev, p.dD, p.B, dA, alpha=p.alpha)
            tkg.gemm_grouped_dev_bf16_wgrad(p.dev, p.dD, p.A, dB, alpha=p.alpha)
    for got, ref in zip(outs, want):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_offsets_past_32_bits():
    # 4.6 GB of gradients and of expert matrices: the last expert's are right
    groups, n, k = 70, 4096, 8192
    sizes = [0] * groups
    sizes[0], sizes[35], sizes[-1] = 20, 0, 37
    dev = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    dD = torch.randn(57, n, generator=g, device="cuda").to(BF16)
    A = torch.randn(57, k, generator=g, device="cuda").to(BF16)
    dB = torch.full((groups, n, k), GUARD, device="cuda", dtype=BF16)
    tkg.gemm_grouped_dev_bf16_wgrad(dev, dD, A, dB)
    assert (dB[35] == 0).all()
    for i, rows in ((0, slice(0, 20)), (groups - 1, slice(20, 57))):
        d, a = dD[rows].to(F64), A[rows].to(F64)
        ref, mag = d.T @ a, d.abs().T @ a.abs()
        within(dB[i], ref, 2.0 ** -7 * ref.abs() + 1e-5 * mag, f"wgrad of expert {i}")
    B = dB
    for i in (0, groups - 1):
        B[i] = torch.randn(n, k, generator=g, device="cuda").to(BF16)
    dA = torch.full((57, k), GUARD, device="cuda", dtype=BF16)
    tkg.gemm_grouped_dev_bf16_dgrad(dev, dD, B, dA)
    for i, rows in ((0, slice(0, 20)), (groups - 1, slice(20, 57))):
        d, b = dD[rows].to(F64), B[i].to(F64)
        ref, mag = d @ b, d.abs() @ b.abs()
        within(dA[rows], ref, 2.0 ** -7 * ref.abs() + 1e-5 * mag, f"dgrad of expert {i}")


def test_refusals():
    p = Groups([10, 20], 64, 128)
    dA, dB = torch.empty(30, 128, device="cuda", dtype=BF16), torch.empty(2, 64, 128, device="cuda", dtype=BF16)
    with pytest.raises(ValueError):
        tkg.gemm_grouped_dev_bf16_dgrad(p.dev.long(), p.dD, p.B, dA)
    with pytest.raises(ValueError):
        tkg.gemm_grouped_dev_bf16_dgrad(p.dev, p.dD, p.B[:1], dA)
    with pytest.raises(ValueError):
        tkg.gemm_grouped_dev_bf16_dgrad(p.dev, p.dD, p.B.transpose(1, 2), dA)
    with pytest.raises(ValueError):
        tkg.gemm_grouped_dev_bf16_wgrad(p.dev, p.dD, p.A, dB, accumulate=True)
    with pytest.raises(ValueError):
        tkg.gemm_grouped_dev_bf16_wgrad(p.dev, p.dD, p.A[:5], dB)
    with pytest.raises(tkg.TkgError) as e:   # 60 columns
        tkg.gemm_grouped_dev_bf16_dgrad(p.dev, p.dD[:, :60].contiguous(), p.B[:, :60].contiguous(), dA)
    assert e.value.status == tkg.ERR_ALIGNMENT


def test_stall_times_out_and_recovers():
    p = Groups([100, 0, 300], 264, 520)
    dA, dB = torch.empty(400, 520, device="cuda", dtype=BF16), torch.empty(3, 264, 520, device="cuda", dtype=BF16)
    try:
        tkg.set_option(tkg.OPT_TIMEOUT_MS, 100)
        tkg.set_option(tkg.OPT_INJECT_STALL, 1)
        tkg.gemm_grouped_dev_bf16_dgrad(p.dev, p.dD, p.B, dA)
        assert tkg.device_status() == tkg.ERR_TIMEOUT
        tkg.gemm_grouped_dev_bf16_wgrad(p.dev, p.dD, p.A, dB)
        assert tkg.device_status() == tkg.ERR_TIMEOUT
    finally:
        tkg.set_option(tkg.OPT_INJECT_STALL, 0)
        tkg.set_option(tkg.OPT_TIMEOUT_MS, 0)
    check_dgrad(p)
    check_wgrad(p)
