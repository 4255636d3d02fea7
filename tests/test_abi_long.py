"""CPU checks of the entry points for long contexts: refusals on the host
before any launch, no-ops on empty work, the binding's checks."""
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


def refuser(lib, fn, names, good):
    def refused(code, text, **over):
        rc = fn(*[dict(good, **over)[n] for n in names])
        assert rc == code, (rc, lib.mla_last_error())
        assert text.encode() in lib.mla_last_error(), lib.mla_last_error()
    return refused


def test_decode_shared_refusals(lib):
    names = ("qa qp cache nb page dtype kv_scale pt mpp pl pr G bt mp sl B qsl T N scale splits out lse ws wsb "
             "stream").split()
    need = lib.mla_decode_shared_workspace_size(4, 2, 8, 16, 0)
    assert need > 0
    assert lib.mla_decode_shared_workspace_size(4, 0, 8, 16, 0) == 0
    assert lib.mla_decode_shared_workspace_size(4, 2, 8, 16, -1) == 0
    good = dict(qa=at(1), qp=at(10), cache=at(100), nb=100, page=64, dtype=0, kv_scale=1.0, pt=at(20), mpp=8, pl=at(21),
                pr=at(22), G=2, bt=at(23), mp=8, sl=at(24), B=4, qsl=at(25), T=8, N=16, scale=0.07, splits=0, out=at(30),
                lse=at(40), ws=at(1000), wsb=need, stream=None)
    refused = refuser(lib, lib.mla_decode_shared, names, good)
    for name in ("B", "T", "G"):
        refused(-1, ">= 0", **{name: -1})
    refused(-1, "at least one prefix", G=0)
    for n in (0, 1025):
        refused(-1, "num_heads", N=n)
    refused(-2, "2^30", T=1 << 26, wsb=1 << 62)
    refused(-2, "<= ", B=(1 << 20) + 1)
    refused(-2, "<= ", G=(1 << 20) + 1)
    for name in ("qa", "qp", "cache", "pt", "pl", "pr", "bt", "sl", "out", "ws"):
        refused(-1, "null", **{name: None})
    refused(-1, "total_q == batch", qsl=None)
    for name in ("qa", "qp", "cache", "out"):
        refused(-1, "aligned", **{name: P(good[name].value + 8)})
    for name in ("pt", "pl", "pr", "bt", "sl", "qsl", "lse"):
        refused(-1, "aligned", **{name: P(good[name].value + 2)})
    refused(-1, "aligned", ws=P((1000 << 20) + 128))
    for page in (0, 8, 100, 512):
        refused(-2, "page_size", page=page)
    refused(-1, "num_blocks", nb=0)
    refused(-1, "num_blocks", nb=1 << 40)
    refused(-1, "max_prefix_pages", mpp=0)
    refused(-1, "max_pages_per_seq", mp=0)
    refused(-2, "2^30", mpp=1 << 25)
    refused(-2, "2^30", mp=1 << 25)
    refused(-2, "too large", T=1 << 18, mp=1 << 18, wsb=1 << 62)
    refused(-2, "too large", T=1 << 18, mpp=1 << 18, wsb=1 << 62)
    refused(-1, "cache_dtype", dtype=2)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        refused(-1, "kv_scale", dtype=1, kv_scale=bad)
    for bad in (0.0, float("nan"), float("inf"), 3e38):
        refused(-1, "scale", scale=bad)
    refused(-1, "num_splits", splits=-1)
    refused(-1, "num_splits", splits=4097)
    refused(-4, "workspace", wsb=need - 1)
    for name in ("qa", "qp", "cache", "pt", "pl", "pr", "bt", "sl", "qsl"):
        refused(-1, "overlap", out=good[name])
        refused(-1, "overlap", lse=good[name])
        refused(-1, "overlap", ws=good[name])
    refused(-1, "overlap", lse=P((30 << 20) + 64))
    refused(-1, "overlap", ws=P((30 << 20) + 256))
    for name in ("B", "T"):
        assert lib.mla_decode_shared(*[dict(good, **{name: 0, "qa": None, "ws": None})[n] for n in names]) == 0


def test_key_weights_refusals(lib):
    names = ("qa qp cache nb page dtype kv_scale bt mp sl B qsl T N scale lse decay w ws wl status stream").split()
    good = dict(qa=at(1), qp=at(10), cache=at(100), nb=100, page=64, dtype=0, kv_scale=1.0, bt=at(23), mp=8, sl=at(24), B=4,
                qsl=at(25), T=8, N=16, scale=0.07, lse=at(40), decay=1.0, w=at(50), ws=600, wl=512, status=at(60), stream=None)
    refused = refuser(lib, lib.mla_key_weights, names, good)
    for name in ("B", "T", "wl"):
        refused(-1, ">= 0", **{name: -1})
    for n in (0, 1025):
        refused(-1, "num_heads", N=n)
    refused(-1, "cache_dtype", dtype=2)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        refused(-1, "kv_scale", dtype=1, kv_scale=bad)
    for bad in (0.0, float("nan"), float("inf"), 3e38, 1e-44):
        refused(-1, "scale", scale=bad)
    for bad in (-0.5, float("nan"), float("inf")):
        refused(-1, "decay", decay=bad)
    refused(-1, "total_q == batch", qsl=None)
    refused(-2, "batch", B=(1 << 20) + 1)
    refused(-2, "page_size", page=48)
    refused(-1, "num_blocks", nb=0)
    refused(-1, "max_pages_per_seq", mp=0)
    refused(-2, "2^30", mp=1 << 25)
    refused(-2, "2^30", T=1 << 26)
    for name in ("qa", "qp", "cache", "bt", "sl", "lse", "w"):
        refused(-1, "null", **{name: None})
    for name in ("qa", "qp", "cache"):
        refused(-1, "aligned", **{name: P(good[name].value + 8)})
    for name in ("bt", "sl", "qsl", "lse", "w", "status"):
        refused(-1, "aligned", **{name: P(good[name].value + 2)})
    refused(-1, "weight_stride", ws=511)
    refused(-1, "weight_stride", ws=(1 << 32) + 1)
    for name in ("qa", "qp", "cache", "bt", "sl", "qsl", "lse"):
        refused(-1, "overlap", w=good[name])
        refused(-1, "overlap", status=good[name])
    refused(-1, "overlap", status=P((50 << 20) + 4))
    assert lib.mla_key_weights(*[dict(good, B=0, T=0, qa=None, w=None)[n] for n in names]) == 0


def test_evict_select_refusals(lib):
    names = "w ws wl sl B budget sinks recent keep lens status stream".split()
    good = dict(w=at(1), ws=1000, wl=1000, sl=at(10), B=4, budget=100, sinks=4, recent=10, keep=at(20), lens=at(30),
                status=at(40), stream=None)
    refused = refuser(lib, lib.mla_evict_select, names, good)
    refused(-1, ">= 0", B=-1)
    refused(-1, ">= 0", wl=-1)
    refused(-1, "budget", budget=0)
    for bad in (dict(sinks=-1), dict(recent=-1), dict(sinks=101), dict(recent=97), dict(recent=2 ** 31 - 1)):
        refused(-1, "sinks", **bad)
    refused(-2, "batch", B=(1 << 20) + 1)
    refused(-2, "2^30", wl=(1 << 30) + 1, ws=1 << 31)
    for name in ("w", "sl", "keep", "lens"):
        refused(-1, "null", **{name: None})
    for name in ("w", "sl", "keep", "lens", "status"):
        refused(-1, "aligned", **{name: P(good[name].value + 2)})
    refused(-1, "weight_stride", ws=999)
    for name in ("w", "sl"):
        refused(-1, "overlap", keep=good[name])
        refused(-1, "overlap", status=good[name])
    refused(-1, "overlap", lens=good["w"])
    refused(-1, "overlap", lens=P((10 << 20) + 4))
    refused(-1, "overlap", lens=good["keep"])
    refused(-1, "overlap", keep=at(10), lens=at(10))
    assert lib.mla_evict_select(*[dict(good, B=0, w=None)[n] for n in names]) == 0


def test_cache_compact_refusals(lib):
    names = "cache nb page dtype bt mp keep mk lens B w ws wl status stream".split()
    good = dict(cache=at(100), nb=100, page=64, dtype=0, bt=at(1), mp=8, keep=at(2), mk=50, lens=at(3), B=4, w=at(4), ws=512,
                wl=512, status=at(5), stream=None)
    refused = refuser(lib, lib.mla_cache_compact, names, good)
    refused(-1, ">= 0", B=-1)
    refused(-1, ">= 0", mk=-1)
    refused(-1, "cache_dtype", dtype=7)
    for name in ("nb", "page", "mp"):
        refused(-1, "positive", **{name: 0})
    refused(-1, "2^31", nb=1 << 25)
    refused(-2, "batch", B=(1 << 20) + 1)
    refused(-2, "2^30", mk=(1 << 30) + 1)
    for name in ("cache", "bt", "keep", "lens"):
        refused(-1, "null", **{name: None})
    refused(-1, "aligned", cache=P((100 << 20) + 8))
    for name in ("bt", "keep", "lens", "w", "status"):
        refused(-1, "aligned", **{name: P(good[name].value + 2)})
    refused(-1, "weight_len", wl=0)
    refused(-1, "weight_stride", ws=511)
    for name in ("bt", "keep", "lens"):
        refused(-1, "overlap", cache=good[name])
        refused(-1, "overlap", w=good[name])
        refused(-1, "overlap", status=good[name])
    refused(-1, "overlap", w=at(100))
    assert lib.mla_cache_compact(*[dict(good, mk=0, cache=None)[n] for n in names]) == 0
    assert lib.mla_cache_compact(*[dict(good, B=0, cache=None)[n] for n in names]) == 0
    assert lib.mla_last_error() == b""


def test_binding_refuses_what_the_library_would_misread(lib):
    import mla_latent_kv_15_gb300 as mla
    i32 = torch.int32
    B, T, N = 2, 2, 4
    q, qp = torch.zeros(T, N, 512, dtype=torch.bfloat16), torch.zeros(T, N, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 64, 576, dtype=torch.bfloat16)
    bt, sl = torch.zeros(B, 2, dtype=i32), torch.zeros(B, dtype=i32)
    pt, pl, pr = torch.zeros(1, 2, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(2, dtype=i32)
    out, lse, ws = torch.zeros(T, N, 512, dtype=torch.bfloat16), torch.zeros(T, N), torch.zeros(10, dtype=torch.uint8)
    w, keep = torch.zeros(B, 100), torch.zeros(B, 10, dtype=i32)

    def shared(**o):
        k = dict(dict(pt=pt, pl=pl, pr=pr), **o)
        mla.decode_shared(q, qp, cache, k["pt"], k["pl"], k["pr"], bt, sl, out, ws, scale=1.0, lse=lse)

    for o in (dict(pl=torch.zeros(2, dtype=i32)), dict(pr=torch.zeros(3, dtype=i32)), dict(pt=pt.long()),
              dict(pt=torch.zeros(2, 4, dtype=i32)[:, ::2]), dict(pr=pr.float())):
        with pytest.raises(ValueError):
            shared(**o)
    with pytest.raises(ValueError, match="CUDA"):
        shared()                       # host tensors

    def weights(**o):
        k = dict(dict(w=w, lse=lse, bt=bt), **o)
        mla.key_weights(q, qp, cache, k["bt"], sl, k["lse"], k["w"], scale=1.0)

    for o in (dict(w=w.double()), dict(w=torch.zeros(3, 100)), dict(w=torch.zeros(B, 200)[:, ::2]), dict(w=torch.zeros(200)),
              dict(lse=lse[:1]), dict(bt=torch.zeros(3, 2, dtype=i32))):
        with pytest.raises(ValueError):
            weights(**o)
    with pytest.raises(ValueError, match="CUDA"):
        weights()
    for o in (dict(keep=keep.long()), dict(keep=keep[:1]), dict(lens=torch.zeros(3, dtype=i32))):
        k = dict(dict(keep=keep, lens=sl), **o)
        with pytest.raises(ValueError):
            mla.evict_select(w, sl, k["keep"], k["lens"])
        with pytest.raises(ValueError):
            mla.cache_compact(cache, bt, k["keep"], k["lens"])
    with pytest.raises(ValueError, match="CUDA"):
        mla.evict_select(w, sl, keep, sl)
    with pytest.raises(ValueError, match="status"):
        mla.cache_compact(cache, bt, keep, sl, status=torch.zeros(2, dtype=i32))
