"""CPU checks that the prompt-side entry points refuse outputs over arguments
they read or write.  The addresses are never dereferenced: every call here is
refused on the host."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from mla_latent_kv_15_gb300 import _build
    import mla_latent_kv_15_gb300 as mla
    _build.build()
    return mla.load()


P = ctypes.c_void_p


def at(mib, more=0):
    return P((mib << 20) + more)


ROPE_NAMES = ("kv_c kvs k_pe pes weight eps positions table max_pos pairs slots T cache nb page dtype kv_scale latent "
              "ls q qts qhs N qo qots qohs status stream").split()
ROPE = dict(kv_c=at(1), kvs=576, k_pe=at(100), pes=64, weight=at(200), eps=1e-6, positions=at(201), table=at(300),
            max_pos=100, pairs=1, slots=at(202), T=8, cache=at(400), nb=10, page=64, dtype=0, kv_scale=1.0,
            latent=at(500), ls=576, q=at(600), qts=20 * 192, qhs=192, N=20, qo=at(700), qots=20 * 64, qohs=64,
            status=at(203), stream=None)


@pytest.mark.parametrize("name,offset", [("weight", 512), ("positions", 32), ("slots", 32), ("table", 25600 - 16),
                                         ("status", 0)])
def test_append_outputs_over_what_all_tokens_read(lib, name, offset):
    def refuse(text, **over):
        rc = lib.mla_rope_cache_write(*[dict(ROPE, **over)[n] for n in ROPE_NAMES])
        assert rc == -1 and text.encode() in lib.mla_last_error(), (rc, lib.mla_last_error())

    there = P(ROPE[name].value + offset)
    refuse("cache must not overlap", cache=there)
    refuse("latent must not overlap", latent=there)
    refuse("q_pe_out must be q_pe", qo=there)
    # one row before it, and a table of unknown size (only its first row is known)
    refuse("q_pe strides", latent=P(ROPE[name].value - 8 * 1152), qts=20)
    refuse("q_pe strides", max_pos=1 << 62, qts=20)


PREFILL_NAMES = "q qts qhs kv kts khs pe pes cu_q cu_kv B T Tk N scale causal splits out lse ws wsb stream".split()


@pytest.mark.parametrize("name,offset", [("q", 100 * 4 * 192 * 2 - 256), ("kv", 256), ("pe", 256), ("cu_q", 0), ("cu_kv", 0),
                                         ("out", 256), ("lse", 1024)])
def test_prefill_outputs_over_other_arguments(lib, name, offset):
    need = lib.mla_prefill_workspace_size(2, 100, 4, 0)
    good = dict(q=at(1), qts=768, qhs=192, kv=at(100), kts=1024, khs=256, pe=at(200), pes=576, cu_q=at(300),
                cu_kv=at(301), B=2, T=100, Tk=500, N=4, scale=0.07, causal=1, splits=0, out=at(400), lse=at(500),
                ws=at(600), wsb=need + (1 << 20), stream=None)

    def refuse(text, **over):
        rc = lib.mla_prefill(*[dict(good, **over)[n] for n in PREFILL_NAMES])
        assert rc in (-1, -4) and text.encode() in lib.mla_last_error(), (rc, lib.mla_last_error())

    there = P(good[name].value + offset)
    if name not in ("out", "lse"):
        refuse("out must not overlap", out=there)
    if name != "lse":
        refuse("lse must not overlap", lse=there)
    refuse("workspace must not overlap", ws=there)
    # right behind the bytes a call needs there may be anything
    refuse("smaller than", lse=P(there.value - 100 * 4 * 4) if name in ("cu_q", "cu_kv") else at(900), wsb=need - 1)
    # without a key, the key tensors are not read
    refuse("smaller than", Tk=0, out=at(100), lse=at(200), wsb=need - 1)


@pytest.mark.parametrize("T,N", [(8, 20), (1, 20), (8, 1)])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("first", [16, 56, -16, -56, 256 - 56])
def test_append_rotated_queries_that_meet_their_source_in_some_columns(lib, T, N, head_major, first):
    """Queries and rotated queries in the same 256-wide rows of heads, `first`
    columns apart: fewer than 64 forwards, backwards or round the row's end."""
    ts, hs = (256, T * 256) if head_major else (N * 256, 256)
    names = dict(qts=ts, qhs=hs, qots=ts, qohs=hs, T=T, N=N, q=at(600, 256), qo=at(600, 256 + 2 * first), latent=None)
    if first > 64 and T * N == 1:
        return                           # one row: behind it lies nothing
    rc = lib.mla_rope_cache_write(*[dict(ROPE, **names)[n] for n in ROPE_NAMES])
    assert rc == -1 and b"q_pe_out must be q_pe" in lib.mla_last_error(), (rc, lib.mla_last_error())
