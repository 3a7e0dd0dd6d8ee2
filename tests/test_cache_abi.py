"""The paged-cache calls refuse out-of-contract arguments on the host, before
anything touches a GPU (CPU only: no compute call is made)."""
import ctypes

import pytest
import torch

import speculative_decoding_drafter_k3_gb300 as k3da
from speculative_decoding_drafter_k3_gb300 import build as kbuild

FAKE = 0x100000  # aligned, never dereferenced: every case fails a host check first
FAR = 1 << 44    # where nothing else overlaps


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return k3da.load_library()


def cache(**over):
    a = dict(pool=FAKE, dtype=k3da.CACHE_BF16, scales=None, pages=16, table=FAKE, stride=4, lens=FAKE, cu=FAKE, R=8)
    a.update({k: v for k, v in over.items() if k in a})
    return list(a.values())


BAD_CACHE = [
    (dict(pool=None), k3da.EINVAL), (dict(pool=FAKE + 8), k3da.EINVAL), (dict(dtype=2), k3da.EINVAL),
    (dict(dtype=-1), k3da.EINVAL), (dict(dtype=k3da.CACHE_E4M3), k3da.EINVAL),       # quantised without scales
    (dict(scales=FAKE), k3da.EINVAL),                                              # bf16 with scales
    (dict(dtype=k3da.CACHE_E4M3, scales=FAKE + 4), k3da.EINVAL),
    (dict(pages=0), k3da.EINVAL), (dict(pages=1 << 40), k3da.EINVAL), (dict(table=None), k3da.EINVAL),
    (dict(table=FAKE + 2), k3da.EINVAL), (dict(stride=0), k3da.EINVAL), (dict(stride=1 << 25), k3da.EINVAL),
    (dict(lens=None), k3da.EINVAL), (dict(cu=None), k3da.EINVAL), (dict(cu=FAKE + 1), k3da.EINVAL),
    (dict(R=0), k3da.EINVAL), (dict(R=1025), k3da.EINVAL), (dict(T=-1), k3da.EINVAL),
    (dict(D=128), k3da.EUNSUPPORTED), (dict(Hkv=0), k3da.EUNSUPPORTED), (dict(Hkv=65, Hq=65), k3da.EUNSUPPORTED),
    (dict(status=FAKE + 2), k3da.EINVAL),
]
BAD_HEADS = [(dict(Hq=7, Hkv=2), k3da.EUNSUPPORTED), (dict(Hq=34, Hkv=2), k3da.EUNSUPPORTED),
             (dict(Hq=0, Hkv=1), k3da.EUNSUPPORTED)]


def append(lib, **over):
    a = dict(qkv=FAR, T=64, Hq=24, Hkv=4, D=64, status=None)
    a.update({k: v for k, v in over.items() if k in a})
    return lib.k3da_kv_append(*cache(**over), a["qkv"], a["T"], a["Hq"], a["Hkv"], a["D"], a["status"], None)


@pytest.mark.parametrize("over,code", BAD_CACHE + BAD_HEADS + [
    (dict(qkv=None), k3da.EINVAL), (dict(qkv=FAR + 2), k3da.EINVAL), (dict(qkv=FAKE + 64), k3da.EINVAL)])
def test_append_refuses(lib, over, code):
    assert append(lib, **over) == code


def append_qknorm(lib, yarn=None, **over):
    a = dict(qkv=FAR, T=64, Hq=24, Hkv=4, D=64, pos=FAKE, pos_dtype=k3da.POS_I32, qw=FAKE, kw=FAKE, eps=1e-5,
             base=1e4, q_out=2 * FAR, status=None)
    a.update({k: v for k, v in over.items() if k in a})
    return lib.k3da_kv_append_qknorm(*cache(**over), a["qkv"], a["T"], a["Hq"], a["Hkv"], a["D"], a["pos"],
                                     a["pos_dtype"], a["qw"], a["kw"], a["eps"], a["base"],
                                     None if yarn is None else ctypes.byref(yarn), a["q_out"], a["status"], None)


@pytest.mark.parametrize("over,code", BAD_CACHE + BAD_HEADS + [
    (dict(qkv=None), k3da.EINVAL), (dict(pos=None), k3da.EINVAL), (dict(pos_dtype=3), k3da.EINVAL),
    (dict(pos=FAKE + 4, pos_dtype=k3da.POS_I64), k3da.EINVAL), (dict(qw=None), k3da.EINVAL), (dict(kw=None), k3da.EINVAL),
    (dict(eps=-1.0), k3da.EINVAL), (dict(eps=float("nan")), k3da.EINVAL), (dict(base=1.0), k3da.EINVAL),
    (dict(q_out=2 * FAR + 8), k3da.EINVAL), (dict(q_out=FAR + 128), k3da.EINVAL), (dict(q_out=FAKE), k3da.EINVAL)])
def test_append_qknorm_refuses(lib, over, code):
    assert append_qknorm(lib, **over) == code


def test_append_qknorm_refuses_bad_yarn(lib):
    assert append_qknorm(lib, yarn=k3da.Yarn.of(0.5, 4096.0)) == k3da.EINVAL


def gather(lib, **over):
    a = dict(k=FAR, v=2 * FAR, T=64, Hkv=4, D=64, status=None)
    a.update({k: v for k, v in over.items() if k in a})
    return lib.k3da_kv_gather(a["k"], a["v"], *cache(**over), a["T"], a["Hkv"], a["D"], a["status"], None)


@pytest.mark.parametrize("over,code", BAD_CACHE + [
    (dict(k=None), k3da.EINVAL), (dict(v=None), k3da.EINVAL), (dict(k=FAR + 2), k3da.EINVAL),
    (dict(v=FAR), k3da.EINVAL), (dict(k=FAKE), k3da.EINVAL)])
def test_gather_refuses(lib, over, code):
    assert gather(lib, **over) == code


def attn(lib, **over):
    a = dict(out=FAR, lse=None, q=2 * FAR, q_stride=24 * 64, T=64, Hq=24, Hkv=4, D=64, mask=0, scale=0.125, ws=FAKE,
             ws_bytes=1 << 40, status=None)
    a.update({k: v for k, v in over.items() if k in a})
    return lib.k3da_chunk_attn(a["out"], a["lse"], a["q"], a["q_stride"], a["T"], *cache(**over), a["Hq"], a["Hkv"],
                               a["D"], a["mask"], a["scale"], a["ws"], a["ws_bytes"], a["status"], None)


@pytest.mark.parametrize("over,code", BAD_CACHE + BAD_HEADS + [
    (dict(out=None), k3da.EINVAL), (dict(q=None), k3da.EINVAL), (dict(out=FAR + 2), k3da.EINVAL),
    (dict(q=2 * FAR + 8), k3da.EINVAL), (dict(lse=FAKE + 2), k3da.EINVAL), (dict(q_stride=24 * 64 - 8), k3da.EINVAL),
    (dict(q_stride=24 * 64 + 4), k3da.EINVAL), (dict(q_stride=(1 << 31) + 8), k3da.EINVAL), (dict(mask=3), k3da.EINVAL),
    (dict(mask=-1), k3da.EINVAL), (dict(scale=0.0), k3da.EINVAL), (dict(scale=float("inf")), k3da.EINVAL),
    (dict(scale=-1.0), k3da.EINVAL), (dict(out=2 * FAR + 64), k3da.EINVAL), (dict(out=FAKE), k3da.EINVAL),
    (dict(ws=None), k3da.EWORKSPACE), (dict(ws=FAKE + 16), k3da.EWORKSPACE), (dict(ws_bytes=64), k3da.EWORKSPACE)])
def test_chunk_attn_refuses(lib, over, code):
    assert attn(lib, **over) == code


def test_chunk_workspace_query(lib):
    ws = lib.k3da_chunk_workspace_bytes
    assert ws(64, 8, 24, 4, 32) > 0 and ws(0, 1, 1, 1, 1) > 0
    for bad in [(-1, 8, 24, 4, 32), (64, 0, 24, 4, 32), (64, 1025, 24, 4, 32), (64, 8, 23, 4, 32), (64, 8, 24, 4, 0),
                (64, 8, 24, 4, 1 << 25), (64, 8, 68, 4, 32)]:
        assert ws(*bad) == 0
        with pytest.raises(k3da.K3daError):
            k3da.chunk_workspace_bytes(*bad)


def test_binding_refuses_host_tensors(lib):
    pool = torch.zeros(2, 2, 1, 64, 64, dtype=torch.bfloat16)
    table, lens, cu = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
    qkv = torch.zeros(1, 8 * 64, dtype=torch.bfloat16)
    with pytest.raises(k3da.K3daError):
        k3da.k3da_kv_append(pool, qkv, table, lens, cu, num_q_heads=6, num_kv_heads=1)
    with pytest.raises(k3da.K3daError):
        k3da.k3da_kv_append_qknorm(pool, qkv, table, lens, cu, torch.zeros(1, dtype=torch.int32), qkv[0, :64], qkv[0, :64],
                                   num_q_heads=6, num_kv_heads=1)
    with pytest.raises(k3da.K3daError):
        k3da.k3da_kv_gather(qkv[:, :64].contiguous(), qkv[:, :64].contiguous(), pool, table, lens, cu, num_kv_heads=1)
    with pytest.raises(k3da.K3daError):
        k3da.k3da_chunk_attn(qkv[:, :384].contiguous(), qkv[:, :384], pool, table, lens, cu, num_q_heads=6,
                             num_kv_heads=1, workspace=torch.zeros(256, dtype=torch.uint8))


def test_quantise_by_the_definition():
    """The tests' own quantiser, at the borders of its rule."""
    from cache_cases import dequantise, quantise
    x = torch.zeros(9, 64, dtype=torch.float64)
    x[0, 0] = 448.0
    x[1, 0] = 449.0                      # over 448: the next power of two
    x[2, 0] = 1.0
    x[3, 0], x[3, 1] = 256.0, 17.0       # 17 = 16 + 1: a tie of step 2, to even -> 16
    x[4, 0], x[4, 1] = 256.0, 19.0       # tie to 20
    x[5, 5] = float("inf")
    x[6, 6] = float("nan")
    x[7, 0], x[7, 1] = 448.0, 2.0 ** -10  # half the smallest code: to 0
    code, byte = quantise(x)
    v = dequantise(code, byte)
    assert byte[:5].tolist() == [127, 128, 119, 127, 127] and byte[5:].tolist() == [255, 255, 127, 0]
    assert v[0, 0] == 448 and v[1, 0] == 448 and v[2, 0] == 1 and v[3, 1] == 16 and v[4, 1] == 20 and v[7, 1] == 0
    assert v[5].isnan().all() and v[6].isnan().all() and (v[8] == 0).all()


def packed(lib, what, args):
    number, count, pack = k3da._PACKED[what]
    return lib.k3da_packed_call(number, pack(*[0 if x is None else x for x in args]), count)


ARGS = {
    "k3da_kv_append": cache() + [FAR, 64, 24, 4, 64, None, None],
    "k3da_kv_append_qknorm": cache() + [FAR, 64, 24, 4, 64, FAKE, k3da.POS_I32, FAKE, FAKE, 1e-5, 1e4, None, 2 * FAR, None,
                                        None],
    "k3da_kv_gather": [FAR, 2 * FAR] + cache() + [64, 4, 64, None, None],
    "k3da_chunk_attn": [FAR, None, 2 * FAR, 24 * 64, 64] + cache() + [24, 4, 64, 0, 0.125, 3 * FAR, 1 << 30, None, None],
}


@pytest.mark.parametrize("what", sorted(ARGS))
def test_a_packed_call_is_the_call(lib, what):
    """Word by word: whatever one argument is changed to, both answer alike.
    (All of them break something first, so that nothing is launched.)"""
    assert len(ARGS[what]) == k3da._PACKED[what][1] == len(getattr(lib, what).argtypes)
    pool = 2 if what == "k3da_kv_gather" else 5 if what == "k3da_chunk_attn" else 0
    base = list(ARGS[what])
    base[pool + 1] = 2  # no cache type
    assert packed(lib, what, base) == getattr(lib, what)(*base) == k3da.EINVAL
    for i, kind in enumerate(getattr(lib, what).argtypes):
        if kind is not ctypes.c_int:
            continue
        for value in (-1, 0, 1 << 30, 4097):
            args = list(ARGS[what])
            args[pool] = FAKE + 8  # a pool that is not aligned
            args[i] = value
            assert packed(lib, what, args) == getattr(lib, what)(*args)
        args = list(ARGS[what])
        args[i] = (1 << 32) + args[i]  # would be right, cut to 32 bits
        assert packed(lib, what, args) == k3da.EINVAL


def test_packed_calls_refuse_what_is_no_call(lib):
    words = bytes(8 * 24)
    for number, count in ((-1, 16), (4, 16), (0, 15), (0, 17), (1, 16), (2, 24), (3, 22)):
        assert lib.k3da_packed_call(number, words, count) == k3da.EINVAL
    assert lib.k3da_packed_call(0, None, 16) == k3da.EINVAL
