"""The operators of a decoding step: exported symbols, the statuses of bad
arguments, the binding's own checks, and the oracle's formulas on hand values.
Runs without a GPU: the addresses are fake and every call but the last ones
carries an error or an empty size."""
import ctypes

import numpy as np
import pytest
import torch

from bit_gemm_block_amd import decode as D
from bit_gemm_block_amd import w4a4 as W
from oracle import decode_oracle as O

P = 0x10000
Q = 0x10002      # aligned to 2 bytes only
S = 0x10004      # aligned to 4 bytes only


@pytest.fixture(scope="module")
def lib():
    return D.lib()


def changed(args, **at):
    bad = list(args)
    for k, v in at.items():
        bad[int(k[1:])] = v
    return bad


def cache(**kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, pages=8, heads=2, page_size=16, head_dim=64, bits=4)
    d.update(kw)
    return ctypes.byref(D.CacheStruct(*(d[n] for n, _ in D.CacheStruct._fields_)))


BAD_CACHES = [dict(pages=0), dict(pages=-1), dict(heads=0), dict(page_size=0), dict(head_dim=0), dict(bits=3),
              dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None)]
UNSUPPORTED_CACHES = [dict(head_dim=96), dict(head_dim=512), dict(page_size=8), dict(page_size=48), dict(page_size=1 << 17),
                      dict(pages=1 << 27), dict(heads=65537)]
MISALIGNED_CACHES = [dict(k=P + 8), dict(v=P + 8), dict(k_scale=S), dict(v_scale=S)]


def test_exports_every_declared_symbol(lib):
    names = D.header_functions()
    assert len(names) == 6
    assert set(names) == set(D._SIGS)
    for n in names:
        assert hasattr(lib, n), n


def test_w4a16_argument_errors(lib):
    f = lib.w4a16_qlinear_forward
    # x dt ldx wq layout ws dt M N K group y dt ldy ws bytes stream
    ok = [P, W.F16, 256, P, W.WEIGHTS_TILED, P, W.F16, 4, 32, 256, 128, P, W.F32, 32, P, 1 << 30, None]
    for bad in (changed(ok, _1=2), changed(ok, _6=-1), changed(ok, _12=7), changed(ok, _2=255), changed(ok, _4=-1),
                changed(ok, _4=4), changed(ok, _7=-1), changed(ok, _8=-1), changed(ok, _9=0), changed(ok, _10=-128),
                changed(ok, _13=31), changed(ok, _0=None), changed(ok, _3=None), changed(ok, _5=None),
                changed(ok, _11=None)):
        assert f(*bad) == W.ERR_INVALID_ARG, bad
    for bad in (changed(ok, _4=W.WEIGHTS_TILED_OB), changed(ok, _4=W.WEIGHTS_TILED_F6), changed(ok, _9=192, _10=0),
                changed(ok, _10=64), changed(ok, _10=384), changed(ok, _9=16512, _2=16512, _10=0),
                changed(ok, _4=W.WEIGHTS_ROWMAJOR, _9=96, _10=0), changed(ok, _4=W.WEIGHTS_ROWMAJOR, _10=32),
                changed(ok, _7=4194241), changed(ok, _8=16776961, _13=16776961)):
        assert f(*bad) == W.ERR_UNSUPPORTED, bad
    for bad in (changed(ok, _0=S), changed(ok, _2=257), changed(ok, _3=S), changed(ok, _5=S), changed(ok, _11=Q),
                changed(ok, _11=P + 1, _12=W.F16)):
        assert f(*bad) == W.ERR_MISALIGNED, bad
    assert f(*changed(ok, _7=0, _0=None)) == W.OK
    assert f(*changed(ok, _8=0, _11=None)) == W.OK
    for bad in ((0, 32, 256), (4, 0, 256), (4, 32, 0), (-1, 32, 256)):
        assert lib.w4a16_qlinear_workspace_size(*bad) == 0


@pytest.mark.parametrize("name", ["w4a4_cache_write", "w4a4_cache_read", "w4a4_cache_attention"])
def test_cache_errors(lib, name):
    f = getattr(lib, name)
    rest = {"w4a4_cache_write": [P, 128, P, 128, W.F16, P, 4, None],
            "w4a4_cache_read": [P, 4, P, 128, P, 128, W.F16, None],
            "w4a4_cache_attention": [P, W.F16, 256, 4, 4, P, 4, 2, P, None, 1, 1, None, 0, None, 0.125, P, W.F16, 256, P,
                                     1 << 30, None]}[name]
    assert f(None, *rest) == W.ERR_INVALID_ARG
    for kw in BAD_CACHES:
        assert f(cache(**kw), *rest) == W.ERR_INVALID_ARG, kw
    for kw in UNSUPPORTED_CACHES:
        assert f(cache(**kw), *rest) == W.ERR_UNSUPPORTED, kw
    for kw in MISALIGNED_CACHES:
        assert f(cache(**kw), *rest) == W.ERR_MISALIGNED, kw


def test_cache_write_and_read_argument_errors(lib):
    f, c = lib.w4a4_cache_write, cache()
    ok = [P, 128, P, 128, W.F16, P, 4, None]
    for bad in (changed(ok, _4=2), changed(ok, _6=-1), changed(ok, _1=127), changed(ok, _3=127), changed(ok, _0=None),
                changed(ok, _2=None), changed(ok, _5=None)):
        assert f(c, *bad) == W.ERR_INVALID_ARG, bad
    for bad in (changed(ok, _0=P + 1), changed(ok, _2=P + 1), changed(ok, _5=Q), changed(ok, _0=Q, _4=W.F32)):
        assert f(c, *bad) == W.ERR_MISALIGNED, bad
    assert f(c, *changed(ok, _6=1 << 28)) == W.ERR_UNSUPPORTED   # 2^32 threads
    assert f(c, *changed(ok, _6=0, _0=None, _5=None)) == W.OK
    f = lib.w4a4_cache_read
    ok = [P, 4, P, 128, P, 128, W.F16, None]
    for bad in (changed(ok, _6=2), changed(ok, _1=-1), changed(ok, _3=127), changed(ok, _5=127), changed(ok, _0=None),
                changed(ok, _2=None, _4=None)):
        assert f(c, *bad) == W.ERR_INVALID_ARG, bad
    for bad in (changed(ok, _2=P + 1), changed(ok, _4=P + 1), changed(ok, _0=Q), changed(ok, _4=Q, _6=W.F32)):
        assert f(c, *bad) == W.ERR_MISALIGNED, bad
    assert f(c, *changed(ok, _1=1 << 28)) == W.ERR_UNSUPPORTED
    assert f(c, *changed(ok, _1=0, _0=None)) == W.OK


def test_attention_argument_errors(lib):
    f, c = lib.w4a4_cache_attention, cache()
    # q dt ldq T Hq tables S width lengths q_start max_q causal ptable pwidth plength scale out dt ldo ws bytes st
    ok = [P, W.F16, 256, 4, 4, P, 4, 2, P, None, 1, 1, None, 0, None, 0.125, P, W.F16, 256, P, 1 << 30, None]
    for bad in (changed(ok, _1=2), changed(ok, _17=2), changed(ok, _2=255), changed(ok, _18=255), changed(ok, _3=-1),
                changed(ok, _4=0), changed(ok, _4=3), changed(ok, _6=-1), changed(ok, _7=-1), changed(ok, _10=0),
                changed(ok, _10=2), changed(ok, _3=3), changed(ok, _13=-1), changed(ok, _12=P), changed(ok, _13=2),
                changed(ok, _12=P, _13=2), changed(ok, _14=P), changed(ok, _15=float("nan")),
                changed(ok, _15=float("inf")), changed(ok, _0=None), changed(ok, _5=None), changed(ok, _8=None),
                changed(ok, _16=None)):
        assert f(c, *bad) == W.ERR_INVALID_ARG, bad
    for bad in (changed(ok, _7=(1 << 26) + 1), changed(ok, _12=P, _13=(1 << 26) + 1, _14=P),
                changed(ok, _3=1 << 30, _6=1 << 30), changed(ok, _9=P, _10=1 << 22, _3=1 << 22)):
        assert f(c, *bad) == W.ERR_UNSUPPORTED, bad
    for bad in (changed(ok, _0=P + 1), changed(ok, _16=P + 1), changed(ok, _5=Q), changed(ok, _8=Q),
                changed(ok, _9=Q), changed(ok, _12=Q, _13=2, _14=P), changed(ok, _12=P, _13=2, _14=Q)):
        assert f(c, *bad) == W.ERR_MISALIGNED, bad
    long = changed(ok, _7=64)                      # parts to be joined
    need = lib.w4a4_cache_attention_workspace_size(c, 4, 4, 4, 64, 1, 0)
    assert need > 0
    assert f(c, *changed(long, _19=None)) == W.ERR_INVALID_ARG
    assert f(c, *changed(long, _19=S)) == W.ERR_MISALIGNED
    assert f(c, *changed(long, _20=need - 1)) == W.ERR_WORKSPACE
    assert f(c, *changed(ok, _3=0, _6=0, _0=None, _16=None)) == W.OK
    assert f(c, *changed(ok, _6=0)) == W.OK
    size = lib.w4a4_cache_attention_workspace_size
    assert size(c, 4, 4, 4, 64, 1, 4) > 0          # a prefix always leaves parts
    for bad in ((4, 3, 4, 64, 1, 0), (-1, 4, 4, 64, 1, 0), (4, 4, 4, -1, 1, 0), (4, 4, 4, 64, 0, 0)):
        assert size(c, *bad) == 0
    assert size(cache(head_dim=80), 4, 4, 4, 64, 1, 0) == 0
    assert size(None, 4, 4, 4, 64, 1, 0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_device_report_unsupported(lib):
    big = 1 << 30
    assert lib.w4a16_qlinear_forward(P, W.F16, 256, P, W.WEIGHTS_TILED, P, W.F16, 4, 32, 256, 128, P, W.F32, 32, P, big,
                                     None) == W.ERR_UNSUPPORTED
    c = cache()
    assert lib.w4a4_cache_write(c, P, 128, P, 128, W.F16, P, 4, None) == W.ERR_UNSUPPORTED
    assert lib.w4a4_cache_read(c, P, 4, P, 128, None, 0, W.F16, None) == W.ERR_UNSUPPORTED
    assert lib.w4a4_cache_attention(c, P, W.F16, 256, 4, 4, P, 4, 2, P, None, 1, 1, None, 0, None, 0.125, P, W.F16, 256,
                                    P, big, None) == W.ERR_UNSUPPORTED


def test_binding_refuses_host_tensors():
    x, i = torch.zeros((4, 128)), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        D.qlinear_w4a16(x, torch.zeros((16, 64), dtype=torch.uint8), torch.zeros(16))
    with pytest.raises(ValueError):
        D.qlinear_w4a16(x, torch.zeros((16, 64), dtype=torch.uint8), torch.zeros(16), w_layout="tiled_ob")
    c = D.KVCache.empty(4, 2, 16, 64, device="cpu")
    assert c.head_dim == 64
    with pytest.raises(ValueError):
        D.cache_write(c, x, x, i)
    with pytest.raises(ValueError):
        D.cache_read(c, i)
    with pytest.raises(ValueError):
        D.cache_attention(x, c, torch.zeros((4, 1), dtype=torch.int32), i)
    with pytest.raises(ValueError):
        D.KVCache.empty(4, 2, 16, 64, bits=5, device="cpu")


def test_oracle_codes_on_hand_values():
    assert O.unpack(np.array([[0x2F, 0x81]], np.uint8), 4).tolist() == [[-1, 2, 1, -8]]
    assert O.unpack(np.array([[0x2F, 0x81]], np.uint8), 8).tolist() == [[47, -127]]
    q = np.array([[-8, 7, 0, -1, 3, -3]])
    assert np.array_equal(O.unpack(O.pack(q, 4), 4), q)
    assert np.array_equal(O.unpack(O.pack(q, 8), 8), q)
    # 3.5 / 1 and 2.5 / 1 lie on a border: ties to even.
    codes, s = O.quantize(np.array([[7.0, 3.5, -2.5, 0.4], [0.0, 0.0, 0.0, 0.0]], np.float32), 4)
    assert codes.tolist() == [[7, 4, -2, 0], [0, 0, 0, 0]] and s.tolist() == [1.0, 0.0]
    codes, s = O.quantize(np.array([[-254.0, 1.0, 3.0, 5.0]], np.float32), 8)
    assert codes.tolist() == [[-127, 0, 2, 2]] and s.tolist() == [2.0]
    w = np.arange(32 * 128, dtype=np.int64).reshape(32, 128).astype(np.uint8)
    t = O.tile(w).reshape(-1)
    # block 1, iteration 1, channels 32 to 63 of the iteration, row 2 of the block
    assert np.array_equal(t[(1 * 2 + 1) * 1024 + (1 * 16 + 2) * 16:][:16], w[18, 64 + 16:64 + 32])


def test_oracle_attention_on_hand_values():
    # Two pages of 16, one head, D = 64; keys and values all zero but channel 0.
    k, v = np.zeros((2, 1, 16, 64)), np.zeros((2, 1, 16, 64))
    k[1, 0, :2, 0] = [1, 2]
    v[1, 0, :2, 0] = [3, 5]
    one = np.ones((2, 1, 16), np.float32)
    c = (O.pack(k, 4), O.pack(v, 4), one, one, 4)
    q = np.zeros((3, 64))
    q[:, 0] = np.log(2.0)                        # scores log 2 and 2 log 2: p = 1/3, 2/3
    out, size, _ = O.attention(q[:1], c, np.array([[1]]), [2], scale=1.0)
    assert np.isclose(out[0, 0], 13 / 3) and out[0, 1] == 0 and np.isclose(size[0, 0], 13 / 3)
    # three queries of a sequence of two tokens: nothing, the first token, both
    out, _, _ = O.attention(q, c, np.array([[1]]), [2], q_start=[0, 3], max_q=3, scale=1.0)
    assert np.allclose(out[:, 0], [0, 3, 13 / 3])
    out, _, _ = O.attention(q, c, np.array([[1]]), [2], q_start=[0, 3], max_q=2, causal=False, scale=1.0)
    assert np.allclose(out[:2, 0], 13 / 3) and np.isnan(out[2]).all()
    # the same two tokens as a prefix: four tokens, p = 1/6, 1/3, 1/6, 1/3
    out, _, _ = O.attention(q[:1], c, np.array([[1]]), [2], scale=1.0, prefix_table=[1], prefix_length=2)
    assert np.isclose(out[0, 0], 13 / 3)
    out, _, _ = O.attention(q[:1], c, np.array([[-1]]), [2], scale=1.0, prefix_table=[1], prefix_length=1)
    assert out[0, 0] == 3
    # a page that does not exist holds nothing; lengths end with the table
    out, _, _ = O.attention(q[:2], c, np.array([[7], [-1]]), [2, 9], scale=1.0)
    assert np.array_equal(out, np.zeros((2, 64)))
    out, _, _ = O.attention(q[:1], c, np.array([[1]]), [99], scale=1.0)
    assert np.isclose(out[0, 0], (2 * 3 + 4 * 5) / (2 + 4 + 14))
