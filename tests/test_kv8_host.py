"""A cache in 8 bits and the token log probabilities answer wrong arguments on the host, without a CUDA call; the 64-bit
definitions of their tests hold on hand-worked cases."""
import ctypes as C

import numpy as np
import pytest

import kv8_util as ref
from test_kv_host import desc


@pytest.fixture(scope="module")
def si():
    import activation_sparse_gb300 as si
    return si


def scales(si, block=1, k=1 << 27, v=1 << 28, k_stride=(1440, 480, 120), v_stride=(1440, 480, 120)):
    s = si.KvScales()
    s.block, s.k, s.v = block, k, v
    s.k_stride[:], s.v_stride[:] = k_stride, v_stride
    return s


def make(si, sc=None, **over):
    h = C.c_void_p()
    sc = scales(si) if sc is None else sc
    rc = si.load().si_kv_create_e4m3(C.byref(desc(si, **over)), C.byref(sc), C.byref(h))
    return rc, h


@pytest.mark.parametrize("over", [
    dict(k=0), dict(v=0), dict(len=0), dict(dtype=2), dict(L=0), dict(B=0), dict(Hkv=0), dict(cap=0), dict(n_slots=0),
    dict(D=8), dict(D=24), dict(D=72), dict(D=264), dict(D=272), dict(k=(1 << 20) + 8), dict(k_stride=(0, 0, 0, 72)),
    dict(v_stride=(8, 0, 0, 64)), dict(k_stride=(0, 0, 0, -64)), dict(table=0, cap=121), dict(n_slots=1 << 31)])
def test_create_refuses(si, over):
    rc, h = make(si, **over)
    assert rc == si.SI_ERR_INVALID_ARG and not h.value
    assert si.load().si_last_error_string()


@pytest.mark.parametrize("over", [dict(block=0), dict(block=-1), dict(block=3), dict(block=48), dict(block=(1 << 30) + 1),
                                  dict(k=0), dict(v=0), dict(k_stride=(-1, 0, 0)), dict(v_stride=(0, 0, -2))])
def test_scales_refuse(si, over):
    rc, h = make(si, sc=scales(si, **over))
    assert rc == si.SI_ERR_INVALID_ARG and not h.value


def test_create(si):
    lib = si.load()
    assert lib.si_kv_create_e4m3(C.byref(desc(si)), None, C.byref(C.c_void_p())) == si.SI_ERR_INVALID_ARG
    assert lib.si_kv_create_e4m3(None, C.byref(scales(si)), C.byref(C.c_void_p())) == si.SI_ERR_INVALID_ARG
    for block in (1, 2, 64, 1 << 30):
        rc, h = make(si, sc=scales(si, block=block))
        assert rc == si.SI_OK and lib.si_kv_destroy(h) == si.SI_OK
    assert make(si, B=1025)[0] == si.SI_ERR_UNSUPPORTED


def test_calls_refuse(si):
    lib = si.load()
    rc, kv = make(si)
    assert rc == si.SI_OK
    p, odd, E = 1 << 20, (1 << 20) + 2, si.SI_ERR_INVALID_ARG
    s3 = (C.c_longlong * 3)(4096, 512, 64)
    rope = si.si_rope_create(64)

    def append(T=2, Hq=8, q=p, k=p, v=p, pos=p, out=p, layer=0):
        return lib.si_kv_append(kv, layer, rope.handle, T, Hq, q, s3, k, s3, v, s3, pos, out, None)

    for over in (dict(k=odd), dict(v=None), dict(q=odd), dict(out=None), dict(T=0), dict(T=101), dict(layer=2), dict(pos=None)):
        assert append(**over) == E, over
    assert lib.si_tree_attention(kv, 0, 65, 8, p, s3, None, 0.1, p + 4096, None, None) == E
    assert lib.si_tree_attention(kv, 0, 2, 6, p, s3, None, 0.1, p + 4096, None, None) == E
    assert lib.si_tree_attention(kv, 0, 2, 8, p, s3, None, 0.1, p, None, None) == E
    assert lib.si_kv_accumulate(kv, 0, 2, 8, p, s3, None, None, None, 0.1, None, None) == E
    assert lib.si_kv_destroy(kv) == si.SI_OK
    none = dict(k_stride=(0, 0, 0, 16), v_stride=(0, 0, 0, 16), table_stride=(0, 0, 0), acc_stride=(0, 0, 0))
    for over, T, G in ((dict(B=1024, Hkv=1024, cap=200000, n_slots=200000), 1, 1),
                       (dict(B=1024, Hkv=1024, cap=64, n_slots=64, D=256), 64, 256),
                       (dict(B=1, Hkv=1, cap=(1 << 31) - 1, n_slots=(1 << 31) - 1), 1, 1)):
        rc, kv = make(si, **over, **none)
        assert rc == si.SI_OK
        Hq = over["Hkv"] * G
        assert lib.si_tree_attention(kv, 0, T, Hq, p, s3, None, 0.1, p + 4096, None, None) == si.SI_ERR_UNSUPPORTED
        assert lib.si_kv_destroy(kv) == si.SI_OK


def test_logprobs_refuse(si):
    lib, p, E = si.load(), 1 << 20, si.SI_ERR_INVALID_ARG

    def call(dtype=0, x=p, stride=100, N=2, V=100, t=1.0, targets=p, M=1, logp=p, entropy=p, K=2, top=p, ids=p):
        return lib.si_token_logprobs(dtype, x, stride, N, V, t, targets, M, logp, entropy, K, top, ids, None)

    for over in (dict(dtype=3), dict(dtype=-1), dict(x=None), dict(x=p + 1), dict(dtype=2, x=p + 2), dict(stride=99), dict(N=-1),
                 dict(V=0), dict(t=0.0), dict(t=-1.0), dict(t=float("nan")), dict(t=float("inf")), dict(t=1e-45), dict(targets=None),
                 dict(logp=None), dict(M=-1), dict(K=-1), dict(K=33), dict(K=5, V=4), dict(top=None), dict(ids=None)):
        assert call(**over) == E, over
    assert call(N=0, x=None) == si.SI_OK                       # nothing to do
    assert call(M=0, K=0, entropy=None) == si.SI_OK


@pytest.mark.parametrize("t", [2.9e-39, 2.95e-39, 3.5e-39, 4.2e-39, 4.239e-39])
def test_logprobs_refuse_a_temperature_whose_exponents_overflow(si, t):
    """1 / t is finite for most of these, log2(e) / t is not."""
    rc = si.load().si_token_logprobs(2, 1 << 20, 100, 2, 100, t, None, 0, None, 1 << 20, 0, None, None, None)
    assert rc == si.SI_ERR_INVALID_ARG and b"temperature" in si.load().si_last_error_string()


@pytest.mark.parametrize("t", [4.25e-39, 1e-38, 1.0, 3.4e38])
def test_logprobs_take_temperatures_to_the_ends(si, t):
    assert si.load().si_token_logprobs(2, None, 100, 0, 100, t, None, 0, None, 1 << 20, 0, None, None, None) == si.SI_OK  # no rows


def test_python_checks(si):
    torch = pytest.importorskip("torch")
    K = torch.zeros(1, 1, 2, 8, 64).to(torch.float8_e4m3fn)
    byte, lens = torch.zeros(1, 1, 2, 8, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_scale and v_scale"):
        si.si_kv_create(K, K, None, lens)
    with pytest.raises(ValueError, match="bf16 or fp16"):
        si.si_kv_create(K, K, None, lens, k_scale=byte, v_scale=byte, dtype=torch.float32)
    H = K.to(torch.bfloat16)
    for extra in (dict(k_scale=byte), dict(block=2), dict(dtype=torch.float16)):
        with pytest.raises(ValueError, match="float8_e4m3fn"):
            si.si_kv_create(H, H, None, lens, **extra)
    x = torch.zeros(2, 5)
    with pytest.raises(ValueError, match="CUDA"):
        si.si_token_logprobs(x)
    with pytest.raises(ValueError, match="bf16, fp16 or fp32"):
        si.si_token_logprobs(x.double())


def test_a_handle_over_16_bits_needs_no_type(si):
    """What wraps a handle by itself need not say what a cache in 16 bits is of."""
    torch = pytest.importorskip("torch")
    K, lens = torch.zeros(1, 1, 2, 8, 64, dtype=torch.float16), torch.zeros(1, 1, dtype=torch.int32)
    kv = si.KV(None, K, K, None, lens, None)
    assert kv.dtype == torch.float16 and kv.block == 1 and kv.k_scale is None and (kv.Hkv, kv.n_slots, kv.cap, kv.D) == (2, 8, 8, 64)


# ------------------------------------------------- the definitions themselves

def test_codes_by_hand():
    assert ref.CODES[0x38] == 1.0 and ref.CODES[0x7E] == 448.0 and ref.CODES[1] == 2.0 ** -9 and ref.CODES[0xB8] == -1.0
    assert np.isnan(ref.CODES[0x7F]) and np.isnan(ref.CODES[0xFF])
    x = np.array([1.0, 1.0625, 1.0626, 1.1875, 447.0, 500.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -9])
    # ties: 1.0625 between 1 and 1.125 to the even fraction, 1.1875 between 1.125 and 1.25, 2^-10 between 0 and 2^-9
    assert ref.CODES[ref.encode(x)].tolist() == [1.0, 1.0, 1.125, 1.25, 448.0, 448.0, -0.0, 0.0, 2 * 2.0 ** -9, -2.0 ** -9]
    for c in range(256):
        if c & 127 != 127:
            assert ref.encode(ref.CODES[c]) == c


def test_scales_by_hand():
    assert ref.scale_byte(448.0, "bf16") == 127 and ref.scale_byte(448.1, "bf16") == 128 and ref.scale_byte(224.0, "fp16") == 126
    assert ref.scale_byte(0.0, "fp16") == 112 and ref.scale_byte(0.0, "bf16") == 3 and ref.scale_byte(np.inf, "bf16") == 255
    assert ref.scale_byte(60000.0, "fp16") == 134 and ref.power(250, "fp16") == 128.0 and np.isnan(ref.power(255, "bf16"))
    # every code stands for a number of the cache's type
    for c in range(127):
        assert np.float16(ref.CODES[c] * 2.0 ** -15) == ref.CODES[c] * 2.0 ** -15
        assert np.float16(ref.CODES[c] * 2.0 ** 7) == ref.CODES[c] * 2.0 ** 7
        assert (ref.CODES[c] * 2.0 ** -124) % 2.0 ** -133 == 0 and ref.CODES[c] * 2.0 ** 119 < 3.39e38


def test_logprobs_by_hand():
    l, h = ref.logprobs(np.log(np.array([[1.0, 3.0], [1.0, 1.0]])), 1.0)
    assert np.allclose(np.exp(l), [[0.25, 0.75], [0.5, 0.5]]) and np.allclose(h, [0.25 * np.log(4) + 0.75 * np.log(4 / 3), np.log(2)])
    l, h = ref.logprobs(np.array([[-np.inf, 0.0], [-np.inf, -np.inf], [np.nan, 0.0], [np.inf, 0.0]]), 2.0)
    assert l[0].tolist() == [-np.inf, 0.0] and h[0] == 0.0
    assert np.isneginf(l[1]).all() and h[1] == 0.0
    assert np.isnan(l[2:]).all() and np.isnan(h[2:]).all()
    assert ref.best(np.array([[1.0, 2.0, 2.0, -0.0, 0.0]]), 5).tolist() == [[1, 2, 0, 3, 4]]
    assert ref.best(np.array([[1.0, np.nan, np.inf, -np.inf]]), 4).tolist() == [[1, 2, 0, 3]]
