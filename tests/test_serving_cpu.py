"""Host checks of sd_cache_append, sd_attend and sd_sample: bad arguments are
refused before any CUDA call, with the reason in the last-error text."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def sd():
    import torch  # noqa: F401  (shares its CUDA runtime with the library)
    import speculative_decoding_verification_sd_gb300 as sd
    sd.build()
    sd._lib.load()
    return sd


P = 1 << 20  # a non-null address that is never dereferenced on these paths


def cache(sd, **kw):
    a = dict(k=P, v=P, page_table=P, k_scale=None, v_scale=None, page_stride=16 * 8 * 64,
             token_stride=8 * 64, head_stride=64, dt=sd.SD_BF16, num_pages=10, page_size=16,
             max_pages=4, heads=8, head_dim=64)
    a.update(kw)
    return sd.sd_kv_cache(**a)


BAD_CACHES = [(dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"),
              (dict(page_table=None), "INVALID_ARG"), (dict(dt=0), "INVALID_ARG"),
              (dict(dt=7), "INVALID_ARG"), (dict(k_scale=P), "INVALID_ARG"),
              (dict(v_scale=P), "INVALID_ARG"), (dict(num_pages=0), "INVALID_ARG"),
              (dict(page_size=0), "INVALID_ARG"), (dict(max_pages=0), "INVALID_ARG"),
              (dict(heads=0), "INVALID_ARG"), (dict(head_dim=4), "UNSUPPORTED"),
              (dict(head_dim=60), "UNSUPPORTED"), (dict(head_dim=264), "UNSUPPORTED"),
              (dict(head_dim=0), "UNSUPPORTED"), (dict(token_stride=-1), "INVALID_ARG")]
BAD_STEPS = [(dict(bs=0), "INVALID_ARG"), (dict(bs=-3), "INVALID_ARG"), (dict(k_max=-1), "INVALID_ARG"),
             (dict(k_max=16), "UNSUPPORTED"), (dict(bs=4097), "UNSUPPORTED"),
             (dict(cu=None), "INVALID_ARG"), (dict(lens=None), "INVALID_ARG"),
             (dict(err=None), "INVALID_ARG"), (dict(c=None), "INVALID_ARG")]


def append(sd, **kw):
    a = dict(kn=P, vn=P, rs=8 * 64, c=cache(sd), cu=P, lens=P, bs=4, k_max=3, err=P)
    a.update(kw)
    c = None if a["c"] is None else ctypes.byref(a["c"])
    return sd._lib.load().sd_cache_append(a["kn"], a["vn"], a["rs"], c, a["cu"], a["lens"], a["bs"],
                                          a["k_max"], a["err"], 0)


def attend(sd, **kw):
    a = dict(q=P, qs=16 * 64, qh=16, c=cache(sd), cu=P, lens=P, bs=4, k_max=3, scale=0.125, out=P,
             lse=None, err=P, ws=P, nb=1 << 40)
    a.update(kw)
    c = None if a["c"] is None else ctypes.byref(a["c"])
    return sd._lib.load().sd_attend(a["q"], a["qs"], a["qh"], c, a["cu"], a["lens"], a["bs"],
                                    a["k_max"], a["scale"], a["out"], a["lse"], a["err"], a["ws"],
                                    a["nb"], 0)


def sample(sd, **kw):
    a = dict(z=P, dt=sd.SD_BF16, V=1024, rows=4, cu=None, bs=4, t=P, k=None, p=None, mp=None, u=P,
             tok=P, kept=None, err=P)
    a.update(kw)
    return sd._lib.load().sd_sample(a["z"], a["dt"], a["V"], a["rows"], a["cu"], a["bs"], a["t"],
                                    a["k"], a["p"], a["mp"], a["u"], a["tok"], a["kept"], a["err"], 0)


@pytest.mark.parametrize("call", [append, attend])
def test_cache_and_step_refusals(sd, call):
    for kw, want in BAD_CACHES:
        assert call(sd, c=cache(sd, **kw)) == getattr(sd, "SD_ERR_" + want), kw
        assert b"no error" not in sd._lib.load().sd_last_error_string()
    for kw, want in BAD_STEPS:
        assert call(sd, **kw) == getattr(sd, "SD_ERR_" + want), kw


def test_append_refusals(sd):
    assert append(sd, kn=None) == sd.SD_ERR_INVALID_ARG
    assert append(sd, vn=None) == sd.SD_ERR_INVALID_ARG
    assert append(sd, rs=8 * 64 - 1) == sd.SD_ERR_SHAPE


def test_attend_refusals(sd):
    assert attend(sd, q=None) == sd.SD_ERR_INVALID_ARG
    assert attend(sd, out=None) == sd.SD_ERR_INVALID_ARG
    assert attend(sd, ws=None) == sd.SD_ERR_INVALID_ARG
    assert attend(sd, ws=P + 128) == sd.SD_ERR_INVALID_ARG
    assert attend(sd, qh=12, qs=12 * 64) == sd.SD_ERR_INVALID_ARG   # 12 heads over 8
    assert attend(sd, qh=0) == sd.SD_ERR_INVALID_ARG
    assert attend(sd, qh=8 * 129, qs=8 * 129 * 64) == sd.SD_ERR_UNSUPPORTED
    assert attend(sd, qs=16 * 64 - 8) == sd.SD_ERR_SHAPE
    assert attend(sd, scale=float("nan")) == sd.SD_ERR_INVALID_ARG
    assert attend(sd, scale=float("inf")) == sd.SD_ERR_INVALID_ARG
    need = sd.sd_attend_workspace_bytes(4, 3, 16, 8, 64)
    assert need > 0 and attend(sd, nb=need - 1) == sd.SD_ERR_SHAPE
    assert b"ws_bytes" in sd._lib.load().sd_last_error_string()
    for bad in ((0, 3, 16, 8, 64), (4, -1, 16, 8, 64), (4, 3, 12, 8, 64), (4, 3, 16, 0, 64), (4, 3, 16, 8, 0)):
        assert sd.sd_attend_workspace_bytes(*bad) == 0


def test_sample_refusals(sd):
    assert sample(sd, dt=sd.SD_E4M3) == sd.SD_ERR_INVALID_ARG
    assert sample(sd, V=0) == sd.SD_ERR_INVALID_ARG
    assert sample(sd, rows=0) == sd.SD_ERR_INVALID_ARG
    assert sample(sd, rows=4096 * 16 + 1) == sd.SD_ERR_UNSUPPORTED
    assert sample(sd, V=sd.SD_MAX_SAMPLE_ROW_BYTES // 2 + 1) == sd.SD_ERR_UNSUPPORTED
    assert sample(sd, dt=sd.SD_F32, V=sd.SD_MAX_SAMPLE_ROW_BYTES // 4 + 1) == sd.SD_ERR_UNSUPPORTED
    assert sample(sd, z=None) == sd.SD_ERR_INVALID_ARG
    assert sample(sd, t=None) == sd.SD_ERR_INVALID_ARG
    assert sample(sd, err=None) == sd.SD_ERR_INVALID_ARG
    assert sample(sd, u=None) == sd.SD_ERR_INVALID_ARG         # tokens without uniforms
    assert sample(sd, tok=None) == sd.SD_ERR_INVALID_ARG       # uniforms without tokens
    assert sample(sd, u=None, tok=None) == sd.SD_ERR_INVALID_ARG   # nothing asked for
    assert sample(sd, cu=P, bs=0) == sd.SD_ERR_INVALID_ARG
    assert sample(sd, z=P + 1) == sd.SD_ERR_INVALID_ARG
    assert sample(sd, kept=P + 1) == sd.SD_ERR_INVALID_ARG


def test_binding_refuses_what_does_not_fit(sd):
    """Shapes, types and host tensors are refused by the Python layer."""
    import torch
    k = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16)
    table = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        sd.KVCache(k, k, table)                      # host tensors
    with pytest.raises(ValueError):
        sd.KVCache(k, k[:2], table)                  # shapes differ
    with pytest.raises(ValueError):
        sd.KVCache(k.float(), k.float(), table)      # dtype
    with pytest.raises(ValueError):
        sd.KVCache(k.transpose(2, 3), k.transpose(2, 3), table)
    with pytest.raises(ValueError):
        sd.KVCache(k, k, table.long())
    z, t = torch.zeros((2, 8)), torch.ones(2)
    with pytest.raises(ValueError):
        sd.sample(z[0], t)                           # not rows
    with pytest.raises(ValueError):
        sd.sample(z, t[:1])                          # too few temperatures
    with pytest.raises(ValueError):
        sd.sample(z, t, top_k=torch.ones(2))         # top_k is int32
    with pytest.raises(ValueError):
        sd.sample(z, t, tokens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        sd.sample(z, t, kept=torch.zeros((2, 7)))
    with pytest.raises(ValueError):
        sd.sample(z.double(), t, kept=True)


def test_options_refusals(sd):
    lib = sd._lib.load()
    nb = sd.sd_attend_workspace_bytes(4, 3, 16, 8, 64)
    c = cache(sd)
    for bad in ((1, 0, 0, 0), (-1, 0, 0, 0), (0, 0x1, 0, 0), (0, 0x40, 0, 0), (0, 0, -1, 0), (0, 0, 0, 1)):
        cfg = ctypes.byref(sd.sd_launch_cfg(*bad))
        assert lib.sd_attend_ex(P, 16 * 64, 16, ctypes.byref(c), P, P, 4, 3, 0.125, P, None, P, P, nb, cfg, 0) == \
            sd.SD_ERR_INVALID_ARG, bad
        assert lib.sd_sample_ex(P, sd.SD_BF16, 1024, 4, None, 4, P, None, None, None, P, P, None, P, cfg, 0) == \
            sd.SD_ERR_INVALID_ARG, bad
        assert b"sd_launch_cfg" in lib.sd_last_error_string()
