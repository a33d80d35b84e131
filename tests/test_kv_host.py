"""The key/value cache's entry points answer wrong arguments on the host,
without a CUDA call; the 64-bit definitions of the tests hold on hand-worked cases."""
import ctypes as C
import math

import numpy as np
import pytest

import kv_util as ref


@pytest.fixture(scope="module")
def si():
    import activation_sparse_gb300 as si
    return si


def desc(si, **over):
    d = si.KvDesc()
    d.dtype, d.L, d.B, d.Hkv, d.D, d.cap, d.n_slots = si.SI_BF16, 2, 3, 4, 64, 100, 120
    d.k = d.v = 1 << 20
    d.k_stride[:] = d.v_stride[:] = (3 * 4 * 120 * 64, 4 * 120 * 64, 120 * 64, 64)
    d.table, d.len, d.acc = 1 << 24, 1 << 25, 1 << 26
    d.table_stride[:] = (3 * 4 * 100, 4 * 100, 100)
    d.acc_stride[:] = (3 * 4 * 120, 4 * 120, 120)
    for name, value in over.items():
        if isinstance(value, tuple):
            getattr(d, name)[:] = value
        else:
            setattr(d, name, value)
    return d


def make(si, **over):
    h = C.c_void_p()
    rc = si.load().si_kv_create(C.byref(desc(si, **over)), C.byref(h))
    return rc, h


@pytest.mark.parametrize("over", [
    dict(k=0), dict(v=0), dict(len=0), dict(dtype=2), dict(L=0), dict(B=0), dict(Hkv=0), dict(cap=0), dict(n_slots=0),
    dict(D=4), dict(D=65), dict(D=264), dict(k=(1 << 20) + 8), dict(k_stride=(0, 0, 0, 60)), dict(v_stride=(4, 0, 0, 64)),
    dict(k_stride=(0, 0, 0, -64)), dict(table=0, cap=121), dict(n_slots=1 << 31), dict(table_stride=(-1, 0, 0))])
def test_create_refuses(si, over):
    rc, h = make(si, **over)
    assert rc == si.SI_ERR_INVALID_ARG and not h.value
    assert si.load().si_last_error_string()


def test_strides_of_single_elements_do_not_matter(si):
    one = dict(L=1, B=1, k_stride=(1, 1, 120 * 64, 64), v_stride=(-3, 1, 120 * 64, 64), table_stride=(1, -1, 100), acc_stride=(-1, 1, 120))
    rc, h = make(si, **one)
    assert rc == si.SI_OK and si.load().si_kv_destroy(h) == si.SI_OK
    assert make(si, **dict(one, B=2))[0] == si.SI_ERR_INVALID_ARG
    rc, h = make(si, L=1, B=1, Hkv=1, cap=1, n_slots=1, k_stride=(1, 1, 1, 1 << 40), v_stride=(1, 1, 1, 1))
    assert rc == si.SI_OK and si.load().si_kv_destroy(h) == si.SI_OK


def test_create_limits(si):
    assert make(si, B=1025)[0] == si.SI_ERR_UNSUPPORTED
    assert si.load().si_kv_create(None, None) == si.SI_ERR_INVALID_ARG
    assert si.load().si_kv_destroy(None) == si.SI_OK
    rc, h = make(si, table=0, cap=120)
    assert rc == si.SI_OK and si.load().si_kv_destroy(h) == si.SI_OK


def test_rope_refuses(si):
    with pytest.raises(si.SIError):
        si.si_rope_create(24, sections=[12])                     # 12 pairs: not whole units of eight
    with pytest.raises(si.SIError):
        si.si_rope_create(64, inv_freq=[float("nan")] * 32)
    with pytest.raises(si.SIError):
        si.si_rope_create(64, inv_freq=[2.0 ** 21] * 32)
    with pytest.raises(si.SIError):
        si.si_rope_create(64, axis=[4] * 32)                     # five axes
    with pytest.raises(si.SIError):
        si.si_rope_create(512)                                   # 256 pairs
    with pytest.raises(ValueError):
        si.si_rope_create(64, sections=[16, 8])
    with pytest.raises(ValueError):
        si.si_rope_create(64, inv_freq=[1.0] * 40)
    r = si.si_rope_create(128, base=500000.0, sections=[16, 24, 24])
    assert (r.n_pairs, r.n_axes) == (64, 3)
    r.close()


def test_calls_refuse(si):
    lib = si.load()
    rc, kv = make(si)
    assert rc == si.SI_OK
    rope = si.si_rope_create(64)
    p, odd = 1 << 20, (1 << 20) + 2
    s3 = (C.c_longlong * 3)(4096, 512, 64)
    bad3 = (C.c_longlong * 3)(4096, 512, 60)
    E = si.SI_ERR_INVALID_ARG

    def append(kv=kv, layer=0, rope=rope.handle, T=2, Hq=8, q=p, qs=s3, k=p, ks=s3, v=p, vs=s3, pos=p, out=p):
        return lib.si_kv_append(kv, layer, rope, T, Hq, q, qs, k, ks, v, vs, pos, out, None)

    for over in (dict(kv=None), dict(rope=None), dict(k=None), dict(v=None), dict(pos=None), dict(q=None), dict(out=None),
                 dict(layer=2), dict(layer=-1), dict(T=0), dict(T=101), dict(Hq=-1), dict(k=odd), dict(v=odd), dict(q=odd),
                 dict(out=odd), dict(ks=bad3), dict(vs=bad3), dict(qs=bad3), dict(ks=None)):
        assert append(**over) == E, over
    wide = si.si_rope_create(128)
    assert append(rope=wide.handle) == E  # 64 pairs exceed D = 64

    def attend(kv=kv, layer=0, T=2, Hq=8, q=p, qs=s3, mask=None, scale=0.125, out=p + 4096, lse=None):
        return lib.si_tree_attention(kv, layer, T, Hq, q, qs, mask, scale, out, lse, None)

    for over in (dict(kv=None), dict(q=None), dict(out=None), dict(qs=None), dict(layer=2), dict(T=0), dict(T=65),
                 dict(Hq=0), dict(Hq=6), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
                 dict(q=odd), dict(out=odd), dict(out=p), dict(qs=bad3)):
        assert attend(**over) == E, over
    assert attend(Hq=4 * 257) == si.SI_ERR_UNSUPPORTED
    rc, small = make(si, cap=1)
    assert attend(kv=small, T=2) == E

    def weigh(kv=kv, lse=p, out=None):
        return lib.si_kv_accumulate(kv, 0, 2, 8, p, s3, lse, None, None, 0.125, out, None)

    assert weigh(kv=None) == E and weigh(lse=None) == E
    rc, no_acc = make(si, acc=0)
    assert weigh(kv=no_acc) == E and b"acc" in lib.si_last_error_string()

    def evict(kv=kv, layer=-1, T=2, path=p, n_path=p, budget=10, sinks=1, recent=2, out=None, len_out=None):
        return lib.si_kv_evict(kv, layer, T, path, n_path, budget, sinks, recent, out, len_out, None)

    for over in (dict(kv=None), dict(kv=no_acc), dict(layer=2), dict(layer=-2), dict(T=-1), dict(T=101), dict(T=65),
                 dict(n_path=None), dict(budget=-1), dict(sinks=-1), dict(recent=-1), dict(sinks=8, recent=3),
                 dict(out=1 << 22), dict(len_out=1 << 22), dict(out=(1 << 24) + 400, len_out=1 << 27),
                 dict(out=1 << 27, len_out=(1 << 25) + 4)):
        assert evict(**over) == E, over
    rc, no_table = make(si, table=0)
    assert evict(kv=no_table) == E
    rc, long_ = make(si, cap=200000, n_slots=200000)
    assert evict(kv=long_) == si.SI_ERR_UNSUPPORTED
    for h in (kv, small, no_acc, no_table, long_):
        assert lib.si_kv_destroy(h) == si.SI_OK


def test_calls_beyond_32_bit_counts_refuse(si):
    """More tiles, lists or units than the kernels' 32-bit counts hold are refused before anything is launched."""
    lib = si.load()
    p, s3 = 1 << 20, (C.c_longlong * 3)(0, 0, 0)
    none = dict(k_stride=(0, 0, 0, 8), v_stride=(0, 0, 0, 8), table_stride=(0, 0, 0), acc_stride=(0, 0, 0))
    rope = si.si_rope_create(64)
    for over, T, G in ((dict(B=1024, Hkv=1024, cap=200000, n_slots=200000), 1, 1),
                       (dict(B=1024, Hkv=1024, cap=64, n_slots=64, D=256), 64, 256),
                       (dict(B=1, Hkv=1, cap=(1 << 31) - 1, n_slots=(1 << 31) - 1), 1, 1)):
        rc, kv = make(si, **over, **none)
        assert rc == si.SI_OK
        Hq = over["Hkv"] * G
        assert lib.si_tree_attention(kv, 0, T, Hq, p, s3, None, 0.1, p + 4096, None, None) == si.SI_ERR_UNSUPPORTED
        if G == 1:
            assert lib.si_kv_accumulate(kv, 0, T, Hq, p, s3, p, None, None, 0.1, None, None) == si.SI_ERR_UNSUPPORTED
        assert lib.si_kv_destroy(kv) == si.SI_OK
    rc, kv = make(si)
    assert lib.si_kv_append(kv, 0, rope.handle, 1, (1 << 31) - 1, p, s3, p, s3, p, s3, p, p, None) == si.SI_ERR_UNSUPPORTED
    assert lib.si_kv_destroy(kv) == si.SI_OK


def test_python_checks(si):
    torch = pytest.importorskip("torch")
    K = torch.zeros(1, 1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        si.si_kv_create(K, K, None, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="bf16 or fp16"):
        si.si_kv_create(K.float(), K.float(), None, torch.zeros(1, 1, dtype=torch.int32))


# ------------------------------------------------- the definitions themselves

def test_angles_against_float64():
    inv = [1.0, 0.1, 1e-3, 500000.0 ** -0.9]
    pos = np.array([[0, 5], [1, -7], [1000, 31]])
    cos, sin = ref.angles(pos, inv, [0, 1, 0, 1])
    want = np.stack([pos[:, 0] * inv[0], pos[:, 1] * inv[1], pos[:, 0] * inv[2], pos[:, 1] * inv[3]], -1)
    assert np.allclose(cos, np.cos(want), atol=2e-13) and np.allclose(sin, np.sin(want), atol=2e-13)
    # one radian per position, far out: sin(2^31 - 1) from a 40-digit value
    c, s = ref.angles(np.array([[2147483647]]), [1.0], [0])
    assert abs(c[0, 0] ** 2 + s[0, 0] ** 2 - 1) < 1e-14
    assert abs(s[0, 0] - math.sin(math.fmod(2147483647.0, 2 * math.pi))) < 1e-6


def test_evict_by_hand():
    table = np.array([[[[5, 0, 3, 1, 4, 2]]]], np.int32)
    acc = np.array([[[[.3, .9, 7., .5, .1, .3]]]])  # by slot
    # live 5 0 3 1, nodes 4 2, node 1 (slot 2) accepted: candidates 5 0 3 1 2 with .3 .3 .5 .9 7
    t, n = ref.evict(table, np.array([[4]], np.int32), acc, 2, np.array([[1, 0]]), np.array([1]), 3, 0, 1)
    assert t[0, 0, 0].tolist() == [3, 1, 2, 5, 0, 4] and n[0, 0] == 3
    t, n = ref.evict(table, np.array([[4]], np.int32), acc, 2, np.array([[1, 0]]), np.array([1]), 4, 0, 0)
    assert t[0, 0, 0].tolist() == [5, 3, 1, 2, 0, 4] and n[0, 0] == 4  # the tie at .3 goes to the earlier candidate
    t, n = ref.evict(table, np.array([[4]], np.int32), acc, 2, None, None, 0, 0, 0)
    assert t[0, 0, 0].tolist() == table[0, 0, 0].tolist() and n[0, 0] == 6


def test_attend_by_hand():
    q = np.ones((1, 1, 1, 2))
    K = np.array([[[[0., 0.], [math.log(3), 0.], [9., 9.]]]])
    V = np.array([[[[4., 0.], [0., 8.], [9., 9.]]]])
    out, lse, _ = ref.attend(q, K, V, None, [1], np.array([[1]], np.uint64), 1.0)
    assert np.allclose(out[0, 0, 0], [1.0, 6.0]) and np.allclose(lse[0, 0, 0], math.log(4))
    out, lse, _ = ref.attend(q, K, V, None, [1], np.array([[0]], np.uint64), 1.0)
    assert not out.any() and np.isneginf(lse).all()
