"""The paged cache's calls refuse bad arguments on the host, before anything reaches a GPU, and the reference that the
GPU tests use agrees with itself.  CPU only."""
import ctypes

import numpy as np
import pytest
import torch

from mamba_ssd_state_b200 import build, dart
from tests import paged_reference as ref

FAKE = ctypes.c_void_p(0x10000)       # 16-byte aligned, never dereferenced on the host
FAR = [ctypes.c_void_p(0x100000000 * (i + 1)) for i in range(16)]
MISALIGNED = ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dart.load()


def cache(**kw):
    f = dict(format=0, npages=8, page_size=4, table_width=3, pages=FAKE, scales=None, table=FAKE)
    f.update(kw)
    return dart.PagedCache(*f.values())


def dims(**kw):
    f = dict(batch=2, seqlen=6, nheads=4, headdim=64, dstate=128, chunk=256, ngroups=1)
    f.update(kw)
    return dart.Dims(*f.values())


def write(lib, d=None, c=None, dtype=1, dH=FAKE, nmem=3, first=FAKE, count=FAKE):
    d, c = d or dims(), cache() if c is None else c
    return lib.dart_cache_write_paged(ctypes.byref(d), dtype, dH, nmem, first, count, ctypes.byref(c), None)


def sma(lib, d=None, c=None, Q=FAKE, y=None, out=FAKE, ws=1 << 30, workspace=FAKE, counts=FAKE):
    d, c = d or dims(), cache() if c is None else c
    return lib.dart_sma_paged(ctypes.byref(d), 1, Q, FAKE, FAKE, FAKE, ctypes.byref(c), counts, 0.5, y, out, workspace, ws, None)


def extend(lib, d=None, c=None, state=FAR[0], state_out=FAR[0], cur=FAR[1], cur_out=FAR[1], n=FAR[2], pos=FAR[3],
           n_out=FAR[4], pos_out=FAR[5], y=FAKE):
    d, c = d or dims(), cache() if c is None else c
    return lib.dart_ssd_extend(ctypes.byref(d), 1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, state, state_out, cur, cur_out,
                               ctypes.byref(c), n, pos, n_out, pos_out, y, FAKE, None)


CALLS = {"write": write, "sma": sma, "extend": extend}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("field, value", [("format", 2), ("format", -1), ("npages", 0), ("page_size", 0), ("table_width", 0),
                                          ("pages", None), ("table", None), ("pages", MISALIGNED), ("table", ctypes.c_void_p(0x10002))])
def test_bad_cache_is_refused(lib, call, field, value):
    assert CALLS[call](lib, c=cache(**{field: value})) == dart.DART_ERR_INVALID_ARG
    assert lib.dart_last_error()


@pytest.mark.parametrize("call", CALLS)
def test_four_bit_pages_need_scales_and_a_compiled_shape(lib, call):
    assert CALLS[call](lib, c=cache(format=1)) == dart.DART_ERR_INVALID_ARG
    assert b"scales" in lib.dart_last_error()
    assert CALLS[call](lib, d=dims(dstate=16, headdim=16), c=cache(format=1, scales=FAKE)) == dart.DART_ERR_UNSUPPORTED
    assert CALLS[call](lib, d=dims(dstate=96)) == dart.DART_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", CALLS)
def test_sizes_out_of_range_are_refused(lib, call):
    assert CALLS[call](lib, c=cache(page_size=1 << 10, table_width=(1 << 9) + 1)) == dart.DART_ERR_UNSUPPORTED
    assert CALLS[call](lib, c=cache(npages=1 << 27, page_size=4)) == dart.DART_ERR_UNSUPPORTED
    assert CALLS[call](lib, d=dims(batch=0)) == dart.DART_ERR_INVALID_ARG
    assert CALLS[call](lib, d=dims(batch=1 << 16)) == dart.DART_ERR_UNSUPPORTED


def test_write_arguments(lib):
    assert write(lib, dtype=7) == dart.DART_ERR_INVALID_ARG
    assert write(lib, nmem=0) == dart.DART_ERR_INVALID_ARG
    for name in ("dH", "first", "count"):
        assert write(lib, **{name: None}) == dart.DART_ERR_INVALID_ARG
        assert name.encode() in lib.dart_last_error()


def test_sma_arguments(lib):
    need = lib.dart_sma_paged_workspace_bytes(ctypes.byref(dims()))
    assert need > 0 and lib.dart_sma_paged_workspace_bytes(None) == 0
    assert sma(lib, ws=need - 1) == dart.DART_ERR_INVALID_ARG
    assert b"workspace" in lib.dart_last_error()
    assert sma(lib, workspace=None) == dart.DART_ERR_INVALID_ARG
    assert sma(lib, Q=None) == dart.DART_ERR_INVALID_ARG
    assert sma(lib, counts=None) == dart.DART_ERR_INVALID_ARG
    assert sma(lib, d=dims(seqlen=-1)) == dart.DART_ERR_INVALID_ARG
    assert sma(lib, d=dims(ngroups=3)) == dart.DART_ERR_INVALID_ARG
    assert sma(lib, y=FAR[0], out=ctypes.c_void_p(FAR[0].value + 4096)) == dart.DART_ERR_INVALID_ARG
    assert b"overlaps" in lib.dart_last_error()
    assert sma(lib, d=dims(seqlen=8 * 4096)) == dart.DART_ERR_UNSUPPORTED
    assert sma(lib, d=dims(seqlen=0), Q=None, out=None, workspace=None) == dart.DART_OK   # nothing to do


def test_extend_arguments(lib):
    assert extend(lib, d=dims(seqlen=-1)) == dart.DART_ERR_INVALID_ARG
    assert extend(lib, y=None) == dart.DART_ERR_INVALID_ARG
    for name in ("state", "state_out", "cur", "cur_out", "n", "pos", "n_out", "pos_out"):
        assert extend(lib, **{name: None}) == dart.DART_ERR_INVALID_ARG
    # the counters after the run have memory of their own
    for kw in (dict(n_out=FAR[2]), dict(pos_out=FAR[2]), dict(pos_out=FAR[3]), dict(n_out=FAR[3])):
        assert extend(lib, **kw) == dart.DART_ERR_INVALID_ARG
        assert b"overlap" in lib.dart_last_error()
    # the state goes onto itself or somewhere else, not onto a part of it, nor onto dH_cur
    for kw in (dict(state_out=ctypes.c_void_p(FAR[0].value + 1024)), dict(state_out=FAR[1]), dict(cur_out=FAR[0])):
        assert extend(lib, **kw) == dart.DART_ERR_INVALID_ARG


def test_results_do_not_go_onto_the_tokens(lib):
    d, c = dims(), cache()
    size = 6 * 4 * 64 * 4
    for k in range(3):                                      # out begins in, and ends in, each of Q, E and Cm
        for off in (64, 16 - size):
            tokens = [FAR[0], FAR[1], FAR[2]]
            out = ctypes.c_void_p(tokens[k].value + off)
            assert lib.dart_sma_paged(ctypes.byref(d), 1, *tokens, FAKE, ctypes.byref(c), FAKE, 0.5, None, out, FAKE, 1 << 30, None) == dart.DART_ERR_INVALID_ARG
            assert b"out overlaps" in lib.dart_last_error()
    for k in (0, 1, 3, 4):                                  # y on x, dt, Bm and Cm
        tokens = [FAR[8], FAR[9], FAR[10], FAR[11], FAR[12]]
        for off in (16, 16 - size):
            y = ctypes.c_void_p(tokens[k].value + off)
            assert lib.dart_ssd_extend(ctypes.byref(d), 1, *tokens, FAKE, FAR[0], FAR[0], FAR[1], FAR[1], ctypes.byref(c), FAR[2], FAR[3],
                                       FAR[4], FAR[5], y, FAKE, None) == dart.DART_ERR_INVALID_ARG
            assert b"y overlaps" in lib.dart_last_error()


EXTEND = ("x", "dt", "A", "Bm", "Cm", "cu_tokens", "state", "state_out", "dH_cur", "dH_cur_out", "n_chunks", "pos", "n_chunks_out",
          "pos_out", "y", "mem_count")
SMA = ("Q", "E", "Cm", "cu_tokens", "mem_count", "y_ssd", "out", "workspace")
CACHE = ("pages", "scales", "table")


def spaced(names):
    return {k: (i + 1) << 34 for i, k in enumerate(names)}          # apart by more than any of them holds


def bytes_of(four_bit):
    """Of every tensor of the calls below: batch 2, 6 tokens, 4 heads, one group, N = 128, P = 64, bfloat16."""
    values = 8 * 4 * 4 * 128 * 64
    ints = dict(cu_tokens=12, n_chunks=8, pos=8, n_chunks_out=8, pos_out=8, mem_count=24, first=8, count=8, table=24)
    return dict(x=3072, dt=96, A=16, Bm=1536, Cm=1536, y=6144, Q=6144, E=3072, y_ssd=6144, out=6144, dH=2 * 4 * 3 * 128 * 64 * 2,
                pages=values // 2 if four_bit else 2 * values, scales=values // 32 if four_bit else 0,
                **dict.fromkeys(("state", "state_out", "dH_cur", "dH_cur_out"), 2 * 4 * 128 * 64 * 4), **ints)


def run_at(lib, call, at, four_bit):
    d = ctypes.byref(dims())
    c = ctypes.byref(cache(format=int(four_bit), pages=at["pages"], scales=at["scales"] if four_bit else None, table=at["table"]))
    p = lambda names: [ctypes.c_void_p(at[k]) for k in names]
    if call == "extend":
        return lib.dart_ssd_extend(d, 1, *p(EXTEND[:10]), c, *p(EXTEND[10:]), None)
    if call == "sma":
        need = lib.dart_sma_paged_workspace_bytes(d)
        return lib.dart_sma_paged(d, 1, *p(SMA[:4]), c, *p(("mem_count",)), 0.5, *p(SMA[5:]), need, None)
    if call == "write":
        return lib.dart_cache_write_paged(d, 1, *p(("dH",)), 3, *p(("first", "count")), c, None)
    return lib.dart_cache_read_paged(d, 1, c, *p(("first", "count", "dH")), 3, None)


RESULTS = {"extend": ("y", "mem_count", "n_chunks_out", "pos_out", "state_out", "dH_cur_out", "pages", "scales"),
           "sma": ("out", "workspace"), "write": ("pages", "scales"), "read": ("dH",)}


@pytest.mark.parametrize("four_bit", [False, True])
@pytest.mark.parametrize("call", RESULTS)
def test_results_have_memory_of_their_own(lib, call, four_bit):
    """Every result against every input and every other result: begun inside it, and ending inside it."""
    names = {"extend": EXTEND + CACHE, "sma": SMA + CACHE, "write": ("dH", "first", "count") + CACHE,
             "read": ("dH", "first", "count", "table")}[call]
    size = dict(bytes_of(four_bit), workspace=lib.dart_sma_paged_workspace_bytes(ctypes.byref(dims())))
    if not four_bit:
        names = tuple(k for k in names if k != "scales")
    for result in RESULTS[call]:
        for other in names:
            # the memories that are moved may lie in the pool as well; scales come with 4-bit pages only
            if result == other or result not in names or (call == "write" and other == "dH"):
                continue
            for at in ((size[other] - 1) // 16 * 16, 16 - -(-size[result] // 16) * 16):
                where = spaced(names + CACHE)
                where[result] = where[other] + at
                assert run_at(lib, call, where, four_bit) == dart.DART_ERR_INVALID_ARG, (result, other, at)
                said = lib.dart_last_error().decode()
                assert f"{result} overlaps {other}" in said or f"{other} overlaps {result}" in said
            if (result, other) not in (("state_out", "state"), ("dH_cur_out", "dH_cur"), ("out", "y_ssd")):
                where = spaced(names + CACHE)
                where[result] = where[other]
                assert run_at(lib, call, where, four_bit) == dart.DART_ERR_INVALID_ARG, (result, other)
    # the one's input in place of the other's is no update in place
    if call == "extend":
        where = spaced(names + CACHE)
        where["state_out"] = where["dH_cur"] = where["state"]
        assert run_at(lib, call, where, four_bit) == dart.DART_ERR_INVALID_ARG


def test_binding_refuses_what_does_not_fit():
    """Checks that need no GPU: they come before the first CUDA call."""
    z = torch.zeros
    with pytest.raises(ValueError):
        dart.dart_cache_write_paged(z(1, 2, 3, 64, 64), z(1), z(1), z(4, 2, 2, 64, 64), z(1, 2))     # host tensors


def test_reference_codes_are_the_nearest_values():
    """Every code midpoint and level goes to the even neighbour, and what is read is within half a step."""
    rng = np.random.default_rng(3)
    V = rng.standard_normal((5, 64, 64)) * np.exp(rng.uniform(-20, 20, (5, 1, 64)))
    V[0, :8, 0] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    V[0, 8:32, 0] = 0.0
    V[1, 3, 2], V[1, 40, 2] = np.nan, np.inf
    codes, scales = ref.quantize(V)
    back = ref.dequantize(codes, scales)
    assert back[0, :8, 0].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]
    assert np.isnan(back[1, :, 2]).all() and np.isfinite(np.delete(back[1], 2, 1)).all()
    fine = np.isfinite(back)
    unit = 2.0 ** (np.repeat(np.moveaxis(scales, -1, -2), 32, -2).astype(float) - 127)
    step = np.where(np.abs(back) / unit < 2, 0.5, np.where(np.abs(back) / unit < 4, 1.0, 2.0))
    assert (np.abs(back - V)[fine] <= (step * unit / 2)[fine]).all()


def test_reference_extend_in_pieces_is_one_run():
    rng = np.random.default_rng(4)
    H, G, N, P, S = 2, 1, 4, 3, 5
    x, Bm, Cm = rng.standard_normal((17, H, P)), rng.standard_normal((17, G, N)), rng.standard_normal((17, G, N))
    dt, A = rng.uniform(0.01, 0.3, (17, H)), -rng.uniform(1, 4, H)
    zero = np.zeros((1, H, N, P))
    whole = ref.extend(x, dt, A, Bm, Cm, [17], zero, zero, [0], [0], S)
    state, cur, n, pos, closed, at = zero, zero, [0], [0], [], 0
    for k in (1, 3, 0, 9, 4):
        y, state, cur, n, pos, counts, app = ref.extend(x[at:at + k], dt[at:at + k], A, Bm[at:at + k], Cm[at:at + k], [k], state,
                                                        cur, n, pos, S)
        np.testing.assert_allclose(y, whole[0][at:at + k], atol=1e-12)
        closed += app[0]
        at += k
    np.testing.assert_allclose(state, whole[1], atol=1e-12)
    np.testing.assert_allclose(closed, whole[6][0], atol=1e-12)
    assert (n, pos) == (whole[3], whole[4]) == ([3], [2])
