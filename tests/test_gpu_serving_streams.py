"""append, attend, sample, plan and verify through their ``stream`` argument
with nothing handed over, and the calls from several host threads."""
import threading

import pytest

import serving_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import speculative_decoding_verification_sd_gb300 as sd  # noqa: E402
from test_gpu_cache_attend import device_cache  # noqa: E402

i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731


def hold(seconds=0.2):
    """Keeps the current stream busy for about that long."""
    torch.cuda._sleep(int(seconds * 2e9))


def attend_inputs(lens=(5000, 20000, 300), counts=(3, 1, 8), seed=0):
    """A step whose segments are cut by the shares' borders."""
    g = torch.Generator().manual_seed(seed)
    k, v, table, _, _ = ref.make_cache(g, list(lens), 16, 2, 128)
    q = torch.randn((len(lens) * 8, 8, 128), generator=g).bfloat16().cuda()
    return q, device_cache(k, v, table, None, None), torch.tensor(ref.compaction(counts)).cuda(), i32(list(lens)), 7


@pytest.fixture(params=["stream", "handle"])
def side(request):
    s = torch.cuda.Stream()
    return s, s if request.param == "stream" else s.cuda_stream


def test_attend_fills_on_the_calls_stream(side):
    s, arg = side
    a = attend_inputs()
    used = int(a[2][-1])
    want = sd.attend(*a, lse=True)
    torch.cuda.synchronize()
    hold()
    r = sd.attend(*a, lse=True, stream=arg)
    torch.cuda.synchronize()
    assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse) and int(r.err) == 0
    assert not r.out[used:].any()
    bad = i32([5000, -1, 300])
    hold()
    r = sd.attend(*a[:3], bad, 7, stream=arg)
    torch.cuda.synchronize()
    assert int(r.err) == sd.SD_DEV_ERR_CACHE


def test_attends_own_workspace_lives_until_the_call_is_done(side):
    s, arg = side
    a = attend_inputs()
    want = sd.attend(*a)
    n = sd.sd_attend_workspace_bytes(3, 7, 8, 2, 128)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        hold()
    r = sd.attend(*a, stream=arg)
    junk = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # a freed workspace's place, if there is one
    torch.cuda.synchronize()
    assert torch.equal(r.out, want.out) and int(r.err) == 0 and int(junk[0]) == 255


def test_append_raises_its_bit_on_the_calls_stream(side):
    _, arg = side
    _, cache, cu, lens, k_max = attend_inputs()
    new, bad = torch.zeros((24, 2, 128), dtype=torch.bfloat16, device="cuda"), i32([5000, -1, 300])
    sd.append(new, new, cache, cu, bad, k_max)  # (loading a kernel would wait for the held stream)
    torch.cuda.synchronize()
    hold()
    err = sd.append(new, new, cache, cu, bad, k_max, stream=arg)
    torch.cuda.synchronize()
    assert int(err) == sd.SD_DEV_ERR_CACHE


def test_sample_fills_on_the_calls_stream(side):
    _, arg = side
    z = torch.randn((9, 5000), generator=torch.Generator().manual_seed(1)).cuda()
    t, u, k = torch.ones(9).cuda(), torch.linspace(0.0, 0.9, 9).cuda(), torch.full((9,), 30, dtype=torch.int32).cuda()
    want = sd.sample(z, t, u, k, kept=True)
    torch.cuda.synchronize()
    assert bool(want.tokens.any())
    hold()
    r = sd.sample(z, t, u, k, kept=True, stream=arg)
    torch.cuda.synchronize()
    assert torch.equal(r.tokens, want.tokens) and torch.equal(r.kept, want.kept) and int(r.err) == 0
    t.neg_()
    torch.cuda.synchronize()
    hold()
    r = sd.sample(z, t, u, stream=arg)
    torch.cuda.synchronize()
    assert int(r.err) == sd.SD_DEV_ERR_TEMP


def test_plan_raises_its_bit_on_the_calls_stream(side):
    _, arg = side
    lens = i32([3, 99, 2])
    sd.plan(lens, 4, mode=sd.SD_MODE_ALL_SLOTS)
    torch.cuda.synchronize()
    hold()
    r = sd.plan(lens, 4, mode=sd.SD_MODE_ALL_SLOTS, stream=arg)
    torch.cuda.synchronize()
    assert int(r.err) == sd.SD_DEV_ERR_DRAFT_LENS


def test_verify_fills_on_the_calls_stream(side):
    _, arg = side
    bs, k, V = 5, 3, 4000
    g = torch.Generator().manual_seed(2)
    z, y = torch.randn((bs * (k + 1), V), generator=g).cuda(), torch.randn((bs * k, V), generator=g).cuda()
    ids, u = torch.randint(0, V, (bs * k,), generator=g).int().cuda(), torch.rand((bs, k + 1), generator=g).cuda()
    cu, t = i32(list(range(0, bs * (k + 1) + 1, k + 1))), torch.ones(bs).cuda()
    want = sd.verify(z, y, sd.SD_F32, V, ids, u, t, cu, k, probs=True)
    torch.cuda.synchronize()
    hold()
    r = sd.verify(z, y, sd.SD_F32, V, ids, u, t, cu, k, probs=True, stream=arg)
    torch.cuda.synchronize()
    assert torch.equal(r.out_tokens, want.out_tokens) and torch.equal(r.accepted_len, want.accepted_len)
    assert torch.equal(torch.nan_to_num(r.probs), torch.nan_to_num(want.probs)) and int(r.err) == 0


def test_inputs_may_be_freed_on_return(side):
    """The memory of an input that the caller lets go of is not handed out again before
    the call's stream has read it."""
    s, arg = side
    q, cache, cu, lens, k_max = attend_inputs()
    g = torch.Generator().manual_seed(6)
    z, t, u = torch.randn((300, 5000), generator=g).cuda(), torch.ones(300).cuda(), torch.rand(300, generator=g).cuda()
    new = torch.randn((24, 2, 128), generator=g).bfloat16().cuda()
    err = i32([0])
    sd.append(new, new, cache, cu, lens, k_max)
    want, wanted = sd.attend(q, cache, cu, lens, k_max), sd.sample(z, t, u)
    k = cache.k.clone()
    cache.k.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        hold()
    sd.append(new.clone(), new.clone(), cache, cu, lens, k_max, stream=arg)
    junk = [torch.full_like(new, 7.0) for _ in range(4)]
    with torch.cuda.stream(s):
        cache.k.copy_(k)
    r = sd.attend(q.clone(), cache, cu, lens, k_max, err=err, stream=arg)
    junk += [torch.full_like(q, 7.0) for _ in range(4)]
    d = sd.sample(z.clone(), t, u, stream=arg)
    junk += [torch.full_like(z, 7.0) for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(r.out, want.out) and int(err) == 0 and torch.equal(d.tokens, wanted.tokens)
    assert all(bool((x == 7.0).all()) for x in junk)


def both(*work, times):
    """Runs the functions in a thread each, on streams of their own; raises what one of them raised."""
    failed, ready = [], threading.Barrier(len(work))

    def loop(fn):
        try:
            s = torch.cuda.Stream()
            ready.wait()
            for _ in range(times):
                fn(s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=loop, args=(fn,)) for fn in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failed:
        raise failed[0]


def test_threads_sample_rows_of_other_lengths():
    """Through the C entry, whose calls run side by side (ctypes lets go of the interpreter)."""
    lib = sd._lib.load()

    def rows(V):
        g = torch.Generator().manual_seed(V)
        z, t, u = torch.randn((1, V), generator=g).cuda(), torch.ones(1).cuda(), torch.rand(1, generator=g).cuda()
        want = sd.sample(z, t, u).tokens.clone()
        got, err = torch.zeros_like(want), torch.zeros(1, dtype=torch.int32, device="cuda")
        at = [x.data_ptr() for x in (z, t, u, got, err)]

        def call(s):
            st = lib.sd_sample(at[0], sd.SD_F32, V, 1, None, 1, at[1], None, None, None, at[2], at[3], None, at[4],
                               s.cuda_stream)
            if st != sd.SD_OK:
                raise AssertionError(f"V={V}: {st} {lib.sd_last_error_string()}")
        return call, got, want, err, z, t, u

    cases = [rows(256000), rows(1000), rows(200000), rows(64)]
    torch.cuda.synchronize()
    both(*(c[0] for c in cases), times=10000)
    for _, got, want, err, *_ in cases:
        assert torch.equal(got, want) and int(err) == 0


def test_threads_attend_with_a_workspace_each():
    def step(seed, lens, counts):
        q, cache, cu, lens, k_max = attend_inputs(lens, counts, seed)
        want = sd.attend(q, cache, cu, lens, k_max).out.clone()
        got, err = torch.zeros_like(want), torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = sd.attend_workspace(cu.numel() - 1, k_max, 8, cache)
        return (lambda s: sd.attend(q, cache, cu, lens, k_max, out=got, err=err, workspace=ws, stream=s)), got, want, err

    a, b = step(1, (5000, 20000, 300), (3, 1, 8)), step(2, (900, 7, 40, 30000), (1, 2, 8, 1))
    torch.cuda.synchronize()
    both(a[0], b[0], times=300)
    for _, got, want, err in (a, b):
        assert torch.equal(got, want) and int(err) == 0


def test_a_captured_call_may_name_its_stream():
    """With nothing handed over, and the capturing stream given as a handle."""
    q, cache, cu, lens, k_max = attend_inputs()
    z = torch.randn((9, 5000), generator=torch.Generator().manual_seed(1)).cuda()
    t, u = torch.ones(9).cuda(), torch.linspace(0.0, 0.9, 9).cuda()
    want, wanted = sd.attend(q, cache, cu, lens, k_max, lse=True), sd.sample(z, t, u, kept=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        at = torch.cuda.current_stream().cuda_stream
        r = sd.attend(q, cache, cu, lens, k_max, lse=True, stream=at)
        d = sd.sample(z, t, u, kept=True, stream=at)
    for _ in range(2):
        for x in (r.out, r.lse, d.tokens, d.kept):
            x.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse) and int(r.err) == 0
        assert torch.equal(d.tokens, wanted.tokens) and torch.equal(d.kept, wanted.kept) and int(d.err) == 0
