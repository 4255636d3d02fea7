"""CPU checks of the prompt-side entry points: refusals on the host before any
launch, no-ops on empty work, the binding's checks."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from mla_latent_kv_15_gb300 import _build
    import mla_latent_kv_15_gb300 as mla
    _build.build()
    return mla.load()


P = ctypes.c_void_p


def at(mib):
    return P(mib << 20)          # addresses that are never dereferenced: validation fails first


def test_rope_cache_write_refusals(lib):
    names = ("kv_c kvs k_pe pes weight eps positions table max_pos pairs slots T cache nb page dtype kv_scale latent "
             "ls q qts qhs N qo qots qohs status stream").split()
    good = dict(kv_c=at(1), kvs=576, k_pe=at(100), pes=64, weight=at(200), eps=1e-6, positions=at(201), table=at(300),
                max_pos=100, pairs=1, slots=at(202), T=8, cache=at(400), nb=10, page=64, dtype=0, kv_scale=1.0,
                latent=at(500), ls=576, q=at(600), qts=20 * 192, qhs=192, N=20, qo=at(700), qots=20 * 64, qohs=64,
                status=at(203), stream=None)

    def refused(code, text, **over):
        rc = lib.mla_rope_cache_write(*[dict(good, **over)[n] for n in names])
        assert rc == code, (rc, lib.mla_last_error())
        assert text.encode() in lib.mla_last_error(), lib.mla_last_error()

    refused(-1, "num_tokens", T=-1)
    refused(-2, "num_tokens", T=8388481)
    refused(-1, "cache_dtype", dtype=2)
    refused(-1, "page_size", page=0)
    refused(-1, "num_blocks", nb=0)
    refused(-1, "num_blocks", nb=1 << 62)
    refused(-1, "max_positions", max_pos=0)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        refused(-1, "kv_scale", dtype=1, kv_scale=bad)
    refused(-1, "norm_eps", eps=-1e-6)
    refused(-1, "norm_eps", eps=float("nan"))
    refused(-1, "together", q=None)
    refused(-1, "together", qo=None)
    refused(-1, "num_heads", N=0)
    refused(-1, "num_heads", N=1025)
    for name in ("kv_c", "k_pe", "positions", "table", "slots", "cache"):
        refused(-1, "null", **{name: None})
    for name in ("kv_c", "k_pe", "table", "cache", "weight", "latent", "q", "qo"):
        refused(-1, "aligned", **{name: P(good[name].value + 8)})
    refused(-1, "aligned", positions=P(good["positions"].value + 4))
    refused(-1, "aligned", status=P(good["status"].value + 2))
    refused(-1, "kv_c_stride", kvs=-8)
    refused(-1, "kv_c_stride", kvs=577)
    refused(-1, "k_pe_stride", pes=(1 << 32) + 8)
    refused(-1, "latent_stride", ls=568)
    refused(-1, "q_pe strides", qts=20)
    refused(-1, "apart", qots=0)
    refused(-1, "apart", qohs=56)
    refused(-1, "apart", qots=64, qohs=64)
    # overlaps
    refused(-1, "cache must not overlap", kv_c=at(400))
    refused(-1, "latent must not overlap", latent=P((1 << 20) + 16))
    refused(-1, "latent must not overlap", latent=at(1), ls=576)          # k_pe is elsewhere: not the input rows
    refused(-1, "latent must not overlap", latent=at(1), k_pe=P((1 << 20) + 1024), pes=640, kvs=640, ls=576)
    refused(-1, "q_pe_out must be q_pe", qo=P((600 << 20) + 128))
    refused(-1, "q_pe_out must be q_pe", qo=at(600), qots=20 * 64, qohs=64)  # other strides than q_pe's
    refused(-1, "q_pe_out must be q_pe", qo=at(400))
    # column ranges of one fused projection's rows are apart: [q of 20 heads | kv_c | k_pe], rotated in place
    base, pitch = 1 << 30, 20 * 192 + 576
    fused = dict(kv_c=P(base + 2 * 20 * 192), kvs=pitch, k_pe=P(base + 2 * (20 * 192 + 512)), pes=pitch,
                 q=P(base + 256), qts=pitch, qhs=192, qo=P(base + 256), qots=pitch, qohs=192, latent=None)
    refused(-1, "q_pe_out must be q_pe", **dict(fused, k_pe=P(base + 2 * 20 * 192 - 16)))
    refused(-2, "num_tokens", **dict(fused, T=8388481))      # (its own layout is accepted: only the size is refused)
    from mla_latent_kv_15_gb300 import MLA_OK
    assert lib.mla_rope_cache_write(*[dict(good, **dict(fused, T=0))[n] for n in names]) == MLA_OK
    # nothing to do
    assert lib.mla_rope_cache_write(*[dict(good, T=0, kv_c=None, cache=None, q=None, qo=None)[n] for n in names]) == 0
    assert lib.mla_last_error() == b""


def test_kv_up_proj_refusals(lib):
    def call(lat=at(1), stride=576, w=at(100), T=8, N=4, D=256, kv=at(200)):
        return lib.mla_kv_up_proj(lat, stride, w, T, N, D, kv, None)

    def refused(code, text, **over):
        assert call(**over) == code
        assert text.encode() in lib.mla_last_error(), lib.mla_last_error()

    refused(-1, "num_tokens", T=-1)
    refused(-2, "num_tokens", T=8388481)
    refused(-1, "num_heads", N=0)
    refused(-1, "num_heads", N=1025)
    for d in (0, 4, 100, 2056):
        refused(-2, "head_dim", D=d)
    refused(-1, "null", w=None)
    refused(-1, "aligned", lat=P((1 << 20) + 8))
    refused(-1, "latent_stride", stride=504)
    refused(-1, "latent_stride", stride=580)
    refused(-1, "overlap", kv=P((1 << 20) + 1024))
    refused(-1, "overlap", kv=at(100))
    assert call(T=0, lat=None, w=None, kv=None) == 0
    assert lib.mla_last_error() == b""


def test_prefill_refusals(lib):
    names = "q qts qhs kv kts khs pe pes cu_q cu_kv B T Tk N scale causal splits out lse ws wsb stream".split()
    need = lib.mla_prefill_workspace_size(2, 100, 4, 0)
    good = dict(q=at(1), qts=768, qhs=192, kv=at(100), kts=1024, khs=256, pe=at(200), pes=576, cu_q=at(300), cu_kv=at(301),
                B=2, T=100, Tk=500, N=4, scale=0.07, causal=1, splits=0, out=at(400), lse=at(500), ws=at(600), wsb=need,
                stream=None)

    def refused(code, text, **over):
        rc = lib.mla_prefill(*[dict(good, **over)[n] for n in names])
        assert rc == code, (rc, lib.mla_last_error())
        assert text.encode() in lib.mla_last_error(), lib.mla_last_error()

    for name in ("B", "T", "Tk"):
        refused(-1, ">= 0", **{name: -1})
    refused(-1, "num_heads", N=0)
    refused(-1, "num_heads", N=1025)
    for bad in (0.0, -0.1, float("nan"), float("inf"), 3e38):
        refused(-1, "scale", scale=bad)
    refused(-1, "num_splits", splits=-1)
    refused(-1, "num_splits", splits=4097)
    refused(-2, "2^30", Tk=(1 << 30) + 1)
    refused(-1, "2^31", T=1 << 30)
    for name in ("q", "kv", "pe", "cu_q", "cu_kv", "out", "ws"):
        refused(-1, "null", **{name: None})
    for name, off in (("q", 8), ("kv", 8), ("pe", 8), ("out", 16)):
        refused(-1, "aligned", **{name: P(good[name].value + off)})
    for name in ("cu_q", "cu_kv", "lse"):
        refused(-1, "aligned", **{name: P(good[name].value + 2)})
    refused(-1, "256-byte", ws=P(good["ws"].value + 128))
    for name in ("qts", "qhs", "kts", "khs", "pes"):
        for bad in (0, -8, 12, (1 << 32) + 8):
            refused(-1, "strides", **{name: bad})
    refused(-1, "overlap", out=P((1 << 20) + 1024))
    refused(-1, "overlap", out=P((100 << 20) + 1024))
    refused(-1, "overlap", out=P((200 << 20) + 1024))
    refused(-4, "workspace", wsb=need - 1)
    refused(-4, "workspace", splits=8)
    refused(-2, "num_splits", T=1 << 20, N=1024, splits=4096, out=at(1 << 20))
    # nothing to do
    assert lib.mla_prefill(*[dict(good, B=0, q=None, out=None, ws=None)[n] for n in names]) == 0
    assert lib.mla_prefill(*[dict(good, T=0, q=None, out=None, ws=None)[n] for n in names]) == 0
    assert lib.mla_last_error() == b""
    assert lib.mla_prefill_status(None, None, None) == -1


def test_prefill_workspace_size(lib):
    f = lib.mla_prefill_workspace_size
    assert f(0, 10, 4, 0) == 0 and f(1, 0, 4, 0) == 0 and f(1, 10, 0, 0) == 0 and f(1, 10, 4, -1) == 0
    assert 0 < f(1, 1, 1, 0) < f(1, 512, 128, 0) <= f(8, 100000, 128, 0) < 200 << 20
    assert f(1, 512, 128, 8) > f(1, 512, 128, 0)


def bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16)


def test_binding_refuses_what_the_append_would_misread():
    import mla_latent_kv_15_gb300 as mla
    T = 6
    down = bf16(T, 576)
    good = dict(kv_c=down[:, :512], k_pe=down[:, 512:], positions=torch.zeros(T, dtype=torch.int64),
                cos_sin=torch.zeros(10, 64), slot_mapping=torch.zeros(T, dtype=torch.int64), cache=bf16(2, 64, 576))

    def call(**over):
        mla.rope_cache_write(**dict(good, **over))

    for text, over in (
            ("kv_c must be bfloat16", dict(kv_c=torch.empty(T, 512))),
            ("kv_c must have shape", dict(kv_c=bf16(T + 1, 512))),
            ("last dimension must be contiguous", dict(kv_c=bf16(512, T).t())),
            ("multiples of 8", dict(kv_c=bf16(T, 580 + 1)[:, :512])),
            ("positions must be int64", dict(positions=torch.zeros(T, dtype=torch.int32))),
            ("cos_sin must be float32", dict(cos_sin=bf16(10, 64))),
            ("cos_sin must have shape", dict(cos_sin=torch.zeros(10, 32))),
            ("slot_mapping must be int64", dict(slot_mapping=torch.zeros(T, dtype=torch.int32))),
            ("norm_weight must have shape", dict(norm_weight=bf16(576))),
            ("latent_out must have shape", dict(latent_out=bf16(T, 512))),
            ("multiples of 8", dict(latent_out=bf16(1, 576).expand(T, -1))),
            ("together", dict(q_pe=bf16(T, 4, 64))),
            ("q_pe_out must have shape", dict(q_pe=bf16(T, 4, 64), q_pe_out=bf16(T, 3, 64))),
            ("status must be int32", dict(status=torch.zeros(1))),
            ("cache rows must be 576", dict(cache=bf16(2, 64, 512))),
            ("CUDA tensor", dict())):
        with pytest.raises(ValueError, match=text):
            call(**over)


def test_binding_refuses_what_the_projection_would_misread():
    import mla_latent_kv_15_gb300 as mla
    for text, lat, w, kv in (
            ("latent must have shape", bf16(5, 576), bf16(2, 256, 512), bf16(5, 2, 256)),
            ("w must have shape", bf16(5, 576)[:, :512], bf16(2, 512, 256), bf16(5, 2, 256)),
            ("w must be contiguous", bf16(5, 512), bf16(2, 512, 512).transpose(1, 2), bf16(5, 2, 512)),
            ("kv must have shape", bf16(5, 512), bf16(2, 256, 512), bf16(5, 256, 2)),
            ("kv must be bfloat16", bf16(5, 512), bf16(2, 256, 512), torch.empty(5, 2, 256)),
            ("CUDA tensor", bf16(5, 512), bf16(2, 256, 512), bf16(5, 2, 256))):
        with pytest.raises(ValueError, match=text):
            mla.kv_up_proj(lat, w, kv)


class _On:
    """Stands for a tensor of some device."""
    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    import mla_latent_kv_15_gb300 as mla
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    mla._on_current_device(_On(0), None, _On(0))
    with pytest.raises(ValueError, match="current device"):
        mla._on_current_device(_On(0), _On(1))
    with pytest.raises(ValueError, match="current device"):
        mla._on_current_device(_On(1), _On(1))


def test_binding_refuses_what_the_prefill_would_misread():
    import mla_latent_kv_15_gb300 as mla
    q, kv, pe = bf16(6, 4, 192), bf16(9, 4, 256), bf16(9, 64)
    cu = torch.tensor([0, 6], dtype=torch.int32)
    ws = torch.empty(1024, dtype=torch.uint8)
    good = dict(q=q, kv=kv, k_pe=pe, cu_q=cu, cu_kv=cu.clone(), out=bf16(6, 4, 128), workspace=ws, scale=0.07)

    def call(**over):
        mla.prefill(**dict(good, **over))

    for text, over in (("q must have shape", dict(q=bf16(6, 4, 128))), ("q must be bfloat16", dict(q=torch.empty(6, 4, 192))),
                       ("kv must have shape", dict(kv=bf16(9, 3, 256))), ("k_pe must have shape", dict(k_pe=bf16(8, 64))),
                       ("multiples of 8", dict(q=bf16(6, 4, 196)[..., :192])),
                       ("last dimension", dict(kv=bf16(9, 256, 4).transpose(1, 2))),
                       ("cu_q must be int32", dict(cu_q=cu.long())), ("cu_kv must have shape", dict(cu_kv=torch.zeros(3, dtype=torch.int32))),
                       ("cu_q must hold", dict(cu_q=torch.zeros(0, dtype=torch.int32))),
                       ("out must have shape", dict(out=bf16(6, 4, 192))), ("out must be contiguous", dict(out=bf16(4, 6, 128).transpose(0, 1))),
                       ("lse must be float32", dict(lse=bf16(6, 4))), ("CUDA tensor", dict())):
        with pytest.raises(ValueError, match=text):
            call(**over)
