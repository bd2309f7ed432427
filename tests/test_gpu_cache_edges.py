"""sd_cache_append and sd_attend at values, scales and lengths that are out of the ordinary.

Tolerances are those of test_gpu_cache_attend.py.
"""
import math

import pytest

import serving_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import speculative_decoding_verification_sd_gb300 as sd  # noqa: E402
from test_gpu_cache_attend import compare, device_cache, run_attend  # noqa: E402

i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
NAN, INF = float("nan"), float("inf")


def attend_with(counts, lens, heads, group, dim, page, e4m3, spoil, seed=0):
    """A step over a cache in which `spoil(k, v, at)` has set elements; at(i, t) = (page, slot)."""
    g = torch.Generator().manual_seed(seed)
    k_max = max(counts) - 1
    k, v, table, ks, vs = ref.make_cache(g, lens, page, heads, dim, e4m3)
    spoil(k, v, lambda i, t: (int(table[i, t // page]), t % page))
    cu = ref.compaction(counts)
    used = int(cu[-1])
    q = torch.randn((len(counts) * (k_max + 1), heads * group, dim), generator=g).bfloat16()
    cache = device_cache(k, v, table, ks, vs)
    r = sd.attend(q.cuda(), cache, torch.tensor(cu).cuda(), i32(lens), k_max, lse=True)
    torch.cuda.synchronize()
    assert int(r.err) == 0
    want, wlse, mass = ref.attend(q[:used], k, v, table, ks, vs, cu, lens, dim ** -0.5)
    out, lse = r.out.cpu()[:used].double(), r.lse.cpu()[:used].double()
    # where the definition is not finite, the same value; elsewhere within the usual bound
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(torch.where(odd, out, 0.0).nan_to_num(nan=0.0), torch.where(odd, want, 0.0).nan_to_num(nan=0.0))
    assert torch.equal(torch.isnan(lse), torch.isnan(wlse))
    only = lambda x: torch.where(odd, 0.0, x)  # noqa: E731
    alive = lambda x: torch.where(torch.isnan(wlse), 0.0, x)  # noqa: E731
    compare(q[:used], k, ks, dim ** -0.5, only(out), alive(lse), only(want), alive(wlse), only(mass))
    return out, want


# a step of four whose own tokens lie in one tile, across two, at the start, and far down a split cache
STEPS = [([4, 1, 3], [100, 50, 3]), ([4, 16, 2], [130, 260, 129]), ([16], [16]), ([5], [30000]), ([5], [29954]), ([8], [129])]


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("dim,heads,group", [(64, 2, 4), (128, 1, 16), (256, 1, 2), (80, 3, 1)])
@pytest.mark.parametrize("counts,lens", STEPS)
def test_a_value_reaches_no_row_that_does_not_see_it(counts, lens, dim, heads, group, page):
    """The last token's values, and those of one in the middle of the step, are not finite
    in some columns: rows before them are as without, rows from them on get the
    definition's infinity or NaN there, and their other columns are untouched."""
    for e4m3 in (False, True):
        def spoil(k, v, at):
            for i, (n, L) in enumerate(zip(counts, lens)):
                if n < 2:
                    continue
                last, mid = at(i, L - 1), at(i, L - n // 2 - 1)
                v[last][0, 3] = NAN if e4m3 else INF
                v[last][0, dim - 1] = NAN
                if not e4m3:
                    v[last][0, 5] = -INF
                    if n > 2:
                        v[mid][0, 5], v[mid][0, 6] = INF, -INF
        out, want = attend_with(counts, lens, heads, group, dim, page, e4m3, spoil)
        assert bool(torch.isfinite(out[0]).all())
        assert not bool(torch.isfinite(want).all())


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_step_of_values_that_are_all_nan(page, e4m3):
    """Every row of the step carries NaN values: the first sees its own, so all are NaN;
    with the first one sound, it alone is finite."""
    for whole in (True, False):
        def spoil(k, v, at):
            for t in range(0 if whole else 1, 6):
                v[at(0, 194 + t)] = NAN
        out, _ = attend_with([6], [200], 2, 8, 128, page, e4m3, spoil)
        assert bool(torch.isnan(out[1:]).all()) and bool(torch.isnan(out[0]).all()) == whole


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_key_reaches_no_row_that_does_not_see_it(page, e4m3):
    for counts, lens in STEPS:
        def spoil(k, v, at):
            for i, (n, L) in enumerate(zip(counts, lens)):
                if n > 1:
                    k[at(i, L - 1)][0, 2] = NAN
        out, _ = attend_with(counts, lens, 2, 4, 128, page, e4m3, spoil)
        assert bool(torch.isfinite(out[0]).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [16, 5])
def test_equal_weights_give_the_mean(page, e4m3):
    """Queries of zeros: every weight is the same power of two and exact in any format,
    so what is left are the fp32 sums (2^-24 a token) and the output's own rounding,
    half a bf16 step of that value.  One token alone gives its own values."""
    g = torch.Generator().manual_seed(7)
    lens, counts = [1, 3, 100, 700, 16], [1, 2, 1, 4, 16]
    k, v, table, ks, vs = ref.make_cache(g, lens, page, 2, 128, e4m3)
    cu = ref.compaction(counts)
    used = int(cu[-1])
    q = torch.zeros((5 * 16, 8, 128), dtype=torch.bfloat16)
    r = sd.attend(q.cuda(), device_cache(k, v, table, ks, vs), torch.tensor(cu).cuda(), i32(lens), 15)
    torch.cuda.synchronize()
    want, _, mass = ref.attend(q[:used], k, v, table, ks, vs, cu, lens, 128 ** -0.5)
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=1e-30))) - 7)
    off = (r.out.cpu()[:used].double() - want).abs()
    assert bool((off <= step / 2 * (1 + 2.0 ** -10) + 700 * 2.0 ** -24 * mass).all()), float((off / step).max())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [16, 5])
def test_weights_keep_more_bits_than_the_output(page, e4m3):
    """Half a bf16 step of the output; of the weights 2^-16 + 2^-18 (two bf16 terms) or
    2^-9 + 2^-11 (a half in three e5m2 terms) and 2^-21 of the exponential; the logits'
    and the sums' fp32 roundings as elsewhere."""
    lens = [2, 3, 5, 9, 20, 130, 700]
    s = run_attend([2] * 7, lens, 2, 4, 128, page, e4m3, seed=11, sharp=1.5)
    k, v, table = s["cache"].k.cpu(), s["cache"].v.cpu(), s["cache"].page_table.cpu()
    ks, vs = (None if x is None else x.cpu() for x in (s["cache"].k_scale, s["cache"].v_scale))
    q = s["q"].cpu()
    want, _, mass = ref.attend(q, k, v, table, ks, vs, s["cu"].cpu(), lens, s["scale"])
    kmax = float(k.float().abs().max()) * (float(ks.max()) if e4m3 else 1.0)
    logit = (128 + 4) * 2.0 ** -24 * q.double().abs().sum(-1)[..., None] * kmax * s["scale"]
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=1e-30))) - 7)
    weight = (2.0 ** -9 + 2.0 ** -11 if e4m3 else 2.0 ** -16 + 2.0 ** -18) + 2.0 ** -21 + 700 * 2.0 ** -24 + 2 * logit
    off = (s["out"].cpu().double() - want).abs()
    assert bool((off <= step / 2 * (1 + 2.0 ** -10) + weight * mass).all()), float((off - weight * mass).div(step).max())


@pytest.mark.parametrize("page", [16, 5])
def test_an_infinite_value_that_all_rows_see(page):
    def spoil(k, v, at):
        v[at(0, 0)][0, 3], v[at(0, 0)][0, 4] = INF, -INF
        v[at(1, 20)][1, 0], v[at(1, 40)][1, 0] = INF, -INF
    out, want = attend_with([3, 4], [300, 129], 2, 4, 64, page, False, spoil)
    assert bool((out[:3, :4, 3] == INF).all()) and bool((out[:3, :4, 4] == -INF).all())
    assert bool(torch.isnan(out[3:, 4:, 0]).all()) and int((~torch.isfinite(out)).sum()) == 3 * 4 * 2 + 4 * 4


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("scale", [0.0, 1e-8, 0.09])
def test_queries_near_the_smallest_normal(scale, e4m3, page):
    """Logits of next to nothing: every visible token weighs the same."""
    g = torch.Generator().manual_seed(4)
    lens, counts = [200, 3], [2, 3]
    k, v, table, ks, vs = ref.make_cache(g, lens, page, 1, 64, e4m3)
    if e4m3:
        ks = torch.full_like(ks, 1e-4)
    for size in (2.0 ** -126, 2.0 ** -133, 2.0 ** -110):
        q = torch.full((6, 4, 64), size).bfloat16()
        cache = device_cache(k, v, table, ks, vs)
        r = sd.attend(q.cuda(), cache, torch.tensor(ref.compaction(counts)).cuda(), i32(lens), 2, scale=scale, lse=True)
        torch.cuda.synchronize()
        want, wlse, mass = ref.attend(q[:5], k, v, table, ks, vs, ref.compaction(counts), lens, scale)
        compare(q[:5], k, ks, scale, r.out.cpu()[:5], r.lse.cpu()[:5], want, wlse, mass)


def test_lengths_next_to_2_to_the_31():
    """One page of 65536 tokens named 32768 times: keys of 0 and values of 1 give
    1 and the logarithm of the length, and longer lengths are cut with their bit."""
    page, most = 65536, sd.SD_MAX_LEN
    k, v = (torch.full((1, page, 1, 8), x, dtype=torch.bfloat16, device="cuda") for x in (0.0, 1.0))
    cache = sd.KVCache(k, v, torch.zeros((1, 2 ** 31 // page), dtype=torch.int32, device="cuda"))
    q = torch.ones((1, 1, 8), dtype=torch.bfloat16, device="cuda")
    for length, bit in ((most, 0), (2 ** 31 - 1, sd.SD_DEV_ERR_CACHE)):
        r = sd.attend(q, cache, i32([0, 1]), i32([length]), 0, lse=True)
        torch.cuda.synchronize()
        assert int(r.err) == bit and bool((r.out == 1).all())
        assert abs(float(r.lse) - math.log(most)) <= 8 * 2.0 ** -22 + 2.0 ** -23 * math.log(most)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim", [136, 160, 192, 72, 248])
def test_head_dims_that_leave_a_column_block_empty(dim, e4m3):
    run_attend([4, 1, 3, 16], [100, 1, 3, 333], 2, 3, dim, 16, e4m3, seed=dim)


@pytest.mark.parametrize("page", [16, 5])
def test_bad_pages_and_lengths_over_an_8_bit_cache(page):
    s = run_attend([1, 2], [40, 60], 2, 2, 64, page, True, k_max=1)
    call = lambda cu=None, lens=None: sd.attend(s["q"], s["cache"], s["cu"] if cu is None else cu,  # noqa: E731
                                                s["lens"] if lens is None else lens, 1, workspace=s["ws"])
    table = s["cache"].page_table
    for bad in (-1, 10 ** 6, s["cache"].num_pages):
        keep = table[1, 1].clone()
        table[1, 1] = bad
        r = call()
        torch.cuda.synchronize()
        assert int(r.err) == sd.SD_DEV_ERR_CACHE
        assert torch.equal(r.out[0], s["out"][0]) and bool(torch.isfinite(r.out).all())
        table[1, 1] = keep
    for length in (-1, 10 ** 9):
        r = call(lens=i32([40, length]))
        torch.cuda.synchronize()
        assert int(r.err) & sd.SD_DEV_ERR_CACHE and torch.equal(r.out[0], s["out"][0])
    for cu in ([0, 3, 4], [0, 1, 0], [-1, 1, 2], [0, 1, 5]):
        r = call(cu=i32(cu))
        torch.cuda.synchronize()
        assert int(r.err) == sd.SD_DEV_ERR_CU_SEQLENS
    r = call()
    torch.cuda.synchronize()
    assert int(r.err) == 0 and torch.equal(r.out[:3], s["out"][:3])


@pytest.mark.parametrize("off", [0, 1])
def test_append_quotients_far_from_one(off):
    """Scales around and beyond 1e-18 and 1e18 and elements around and beyond 2^59: the
    fp32 quotient, rounded to e4m3, bit for bit."""
    scales = torch.tensor([1e-18, 1.0000001e-18, 9.99e-19, 1e-30, 3e-39, 1e18, 9.9999997e17, 1.01e18, 1e30, 3e38, 0.02, 1.0])
    x = torch.tensor([2.0 ** 59, 2.0 ** 59 * 0.99609375, 2.0 ** 60, 3e38, 1e-38, 1e-40, 0.0, -1.0, -(2.0 ** 59), 447.0,
                      1e-18, -3e-17, 2e18, 4.4e20, -1e9, 0.019])
    heads, dim = len(scales), 16
    new = x.bfloat16().view(1, 1, dim).expand(1, heads, dim).contiguous()
    k, v = (torch.zeros((1, 4 * heads * dim + off), dtype=torch.uint8, device="cuda")[:, off:]
            .view(torch.float8_e4m3fn).unflatten(1, (4, heads, dim)) for _ in range(2))
    cache = sd.KVCache(k, v, i32([[0]]), k_scale=scales.cuda(), v_scale=scales.cuda())
    err = sd.append(new.cuda(), new.cuda(), cache, i32([0, 1]), i32([3]), 0)
    torch.cuda.synchronize()
    assert int(err) == 0
    want = (new[0].float() / scales[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for got in (k, v):
        assert torch.equal(got[0, 2].view(torch.uint8).cpu(), want)
        assert not got[0, [0, 1, 3]].view(torch.uint8).any()


def test_sample_leaves_every_row_of_an_invalid_range_alone():
    z = torch.randn((8, 512), generator=torch.Generator().manual_seed(4)).cuda()
    for cu in ([0, -2], [5, 3], [0, 9], [4, 2, 3]):
        kept = torch.full_like(z, 77.0)
        tokens = torch.full((8,), -5, dtype=torch.int32, device="cuda")
        r = sd.sample(z, torch.ones(2).cuda(), torch.full((8,), 0.5).cuda(), tokens=tokens, kept=kept, cu_seqlens=i32(cu))
        torch.cuda.synchronize()
        assert int(r.err) == sd.SD_DEV_ERR_CU_SEQLENS
        live = [2] if cu == [4, 2, 3] else []
        rest = [row for row in range(8) if row not in live]
        assert bool((kept[rest] == 77.0).all()) and bool((tokens[rest] == -5).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [16, 24, 5])
def test_a_prompt_goes_in_as_requests_that_share_its_pages(page, e4m3):
    g = torch.Generator().manual_seed(8)
    heads, dim, tokens = 2, 64, 100
    k, v, table, ks, vs = ref.make_cache(g, [tokens], page, heads, dim, e4m3)
    new = torch.randn((112, 2, heads, dim), generator=g).bfloat16()
    counts = [16] * 6 + [4]
    cache = device_cache(k, v, table.repeat(7, 1), ks, vs)
    nd = new.cuda()
    ends = torch.tensor(counts).cumsum(0).tolist()
    err = sd.append(nd[:, 0], nd[:, 1], cache, torch.tensor(ref.compaction(counts)).cuda(), i32(ends), 15)
    torch.cuda.synchronize()
    assert int(err) == 0
    t = torch.arange(tokens)
    at = table[0, t // page].long(), t % page
    for w, (x, sc) in enumerate(((k, ks), (v, vs))):
        y = new[:tokens, w]
        y = (y.float() / sc[:, None]).clamp(-448, 448).to(x.dtype) if e4m3 else y
        for i in range(tokens):
            x[at[0][i], at[1][i]] = y[i]
        got = (cache.v if w else cache.k).cpu()
        assert torch.equal(got.view(torch.uint8), x.contiguous().view(torch.uint8))
