"""Device-side waits of sd_attend and sd_sample that run out (the test hook loads
nothing): the kernels return, raise their bit, and the next call is right."""
import pytest

import serving_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import speculative_decoding_verification_sd_gb300 as sd  # noqa: E402
from test_gpu_cache_attend import device_cache  # noqa: E402

STALL = {"flags": sd.SD_TEST_STALL, "wait_limit_us": 20000}
i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731


@pytest.mark.parametrize("e4m3", [False, True])
def test_attend_gives_up_and_goes_on(e4m3):
    g = torch.Generator().manual_seed(3)
    lens, k_max = [5000, 9000, 300], 7
    k, v, table, ks, vs = ref.make_cache(g, lens, 16, 2, 128, e4m3)
    cache = device_cache(k, v, table, ks, vs)
    q = torch.randn((24, 8, 128), generator=g).bfloat16().cuda()
    cu, lens = torch.tensor(ref.compaction([3, 1, 8])).cuda(), i32(lens)
    ws = sd.attend_workspace(3, k_max, 8, cache)
    want = sd.attend(q, cache, cu, lens, k_max, lse=True, workspace=ws)
    torch.cuda.synchronize()
    out, lse, err = torch.zeros_like(want.out), torch.zeros_like(want.lse), i32([0])
    call = lambda cfg: sd.sd_attend_ex(q, 8 * 128, 8, cache, cu, lens, 3, k_max, 128 ** -0.5, out, lse, err,  # noqa: E731
                                       ws, ws.numel(), cfg=cfg)
    call(STALL)
    torch.cuda.synchronize()
    assert int(err) == sd.SD_DEV_ERR_TIMEOUT
    assert not out[12:].any() and not lse[12:].any()
    ws.zero_()
    err.zero_()
    call({"wait_limit_us": 500000})
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(out, want.out) and torch.equal(lse, want.lse)
    assert not ws[:640].any()


@pytest.mark.parametrize("dtype,V", [(torch.float32, 4096), (torch.bfloat16, 129280)])
def test_sample_gives_up_and_goes_on(dtype, V):
    z = torch.randn((3, V), generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    t, u, k = torch.ones(3).cuda(), torch.tensor([0.3, 0.6, 0.9]).cuda(), i32([0, 40, 3000])
    want = sd.sample(z, t, u, k, kept=True)
    kept, tokens, err = torch.full_like(z, 77.0), i32([-5, -5, -5]), i32([0])
    torch.cuda.synchronize()
    call = lambda cfg: sd.sd_sample_ex(z, z.dtype, V, 3, None, 3, t, k, None, None, u, tokens, kept, err, cfg=cfg)  # noqa: E731
    call(STALL)
    torch.cuda.synchronize()
    assert int(err) & sd.SD_DEV_ERR_TIMEOUT
    assert not tokens.any() and bool((kept == 77.0).all())
    err.zero_()
    call(None)
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(tokens, want.tokens) and torch.equal(kept, want.kept)
