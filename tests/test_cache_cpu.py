"""Host-side refusals of the operators over a cache of 8-bit rows: every call below fails its checks before anything is
launched, so no GPU is needed."""
import ctypes

import pytest
import torch

import plain64_cache as pc
from speculative_decoding_verification_verify_gb300 import _build, binding, binding_cache

A, ODD, ODD4 = 0x10000, 0x10008, 0x10002  # never dereferenced
E = binding.E4M3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load_library()


def append(lib, **bad):
    a = dict(q=A, k=A, v=A, dtype=0, qs=48 * 128, ks=48 * 128, vs=48 * 128, q_out=A, kc=A, vc=A, cache=E, slots=100,
             kss=1040, vss=1040, table=A, max_pos=64, committed=A, parents=None, num_nodes=None, cs=A, positions=64, rot=128,
             interleaved=0, qn=A, kn=A, eps=1e-6, B=2, N=8, Hq=32, Hkv=8, D=128, status=None, stream=None)
    assert set(bad) <= set(a)
    return lib.spec_verify_kv_append_ex(*{**a, **bad}.values())


def test_append(lib):
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(q_out=None), dict(kc=None), dict(vc=None),
                dict(table=None), dict(committed=None), dict(dtype=1), dict(dtype=E), dict(cache=1), dict(cache=2),
                dict(cache=4), dict(B=0), dict(N=0), dict(parents=A, N=65), dict(max_pos=0), dict(slots=0),
                dict(slots=1 << 31), dict(Hq=0), dict(Hkv=0), dict(D=120), dict(D=8), dict(D=528), dict(rot=8),
                dict(rot=144), dict(rot=-16), dict(cs=None), dict(positions=0), dict(qs=32 * 128 - 8), dict(qs=48 * 128 + 4),
                dict(ks=1016), dict(vs=1016), dict(kss=1024), dict(vss=1048), dict(vss=-1040), dict(cache=0, kss=1016),
                dict(cache=0, vss=1036), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(q_out=ODD), dict(kc=ODD),
                dict(vc=ODD), dict(cs=ODD), dict(qn=ODD), dict(kn=ODD), dict(eps=-1e-6), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(table=ODD4), dict(committed=ODD4), dict(parents=ODD4), dict(num_nodes=ODD4),
                dict(status=ODD4), dict(B=1 << 16, N=1 << 16), dict(q=A, q_out=A + 16)):
        assert append(lib, **bad) == binding.EINVAL, bad


def read(lib, **bad):
    a = dict(kc=A, vc=A, cache=E, slots=100, kss=1040, vss=1040, table=A, max_pos=64, first=A, num=None, B=2, N=8, Hkv=8,
             D=128, k_out=A, v_out=A, dtype=0, status=None, stream=None)
    assert set(bad) <= set(a)
    return lib.spec_verify_kv_read(*{**a, **bad}.values())


def test_read(lib):
    for bad in (dict(kc=None), dict(vc=None), dict(table=None), dict(first=None), dict(k_out=None), dict(v_out=None),
                dict(cache=1), dict(cache=2), dict(dtype=1), dict(dtype=E), dict(slots=0), dict(slots=1 << 31),
                dict(kss=1024), dict(vss=1048), dict(max_pos=0), dict(B=0), dict(N=0), dict(B=1 << 16, N=1 << 16),
                dict(Hkv=0), dict(D=8), dict(D=24), dict(D=528), dict(kc=ODD), dict(vc=ODD), dict(k_out=ODD),
                dict(v_out=ODD), dict(k_out=A + 16), dict(v_out=A + 16), dict(table=ODD4), dict(first=ODD4), dict(num=ODD4), dict(status=ODD4)):
        assert read(lib, **bad) == binding.EINVAL, bad


def nodes(lib, **bad):
    a = dict(q=A, dtype=0, qs=32 * 128, kc=A, vc=A, slots=100, kss=1040, vss=1040, table=A, max_pos=64, committed=A,
             parents=None, num_nodes=None, B=2, N=8, Hq=32, Hkv=8, D=128, scale=0.1, out=A, lse=None, ws=A,
             nbytes=1 << 30, status=None, stream=None)
    assert set(bad) <= set(a)
    return lib.spec_verify_attention_e4m3(*{**a, **bad}.values())


def test_nodes(lib):
    for bad in (dict(q=None), dict(kc=None), dict(vc=None), dict(table=None), dict(committed=None), dict(out=None),
                dict(ws=None), dict(dtype=1), dict(dtype=E), dict(B=0), dict(B=65537), dict(N=0), dict(N=65), dict(Hq=0),
                dict(Hkv=0), dict(Hkv=5), dict(D=48), dict(D=72), dict(D=144), dict(max_pos=0), dict(slots=0),
                dict(slots=1 << 31), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(qs=4088),
                dict(kss=1024), dict(vss=1048), dict(kss=1 << 31), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD),
                dict(table=ODD4), dict(committed=ODD4), dict(parents=ODD4), dict(num_nodes=ODD4), dict(lse=ODD4),
                dict(status=ODD4)):
        assert nodes(lib, **bad) == binding.EINVAL, bad
    assert nodes(lib, nbytes=16) == binding.EWORKSPACE
    assert nodes(lib, ws=0x10080) == binding.EWORKSPACE


def chunk(lib, **bad):
    a = dict(q=A, dtype=0, qs=32 * 128, kc=A, vc=A, cache=E, slots=100, kss=1040, vss=1040, table=A, max_pos=64,
             committed=A, num_nodes=None, B=2, N=800, Hq=32, Hkv=8, D=128, scale=0.1, out=A, lse=None, ws=A,
             nbytes=1 << 30, status=None, stream=None)
    assert set(bad) <= set(a)
    return lib.spec_verify_attention_chunk(*{**a, **bad}.values())


def test_chunk(lib):
    for bad in (dict(q=None), dict(kc=None), dict(vc=None), dict(table=None), dict(committed=None), dict(out=None),
                dict(ws=None), dict(dtype=1), dict(dtype=E), dict(cache=1), dict(cache=2), dict(cache=-1), dict(B=0),
                dict(B=65537), dict(N=0), dict(B=65536, N=65536), dict(Hq=0), dict(Hkv=0), dict(Hkv=5), dict(D=48),
                dict(D=72), dict(D=144), dict(max_pos=0), dict(max_pos=(1 << 31) - 1), dict(slots=0), dict(slots=1 << 31),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(qs=4088),
                dict(qs=4100), dict(kss=1024), dict(vss=1048), dict(kss=1 << 31), dict(cache=0, kss=1016),
                dict(cache=0, vss=1028), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD), dict(table=ODD4),
                dict(committed=ODD4), dict(num_nodes=ODD4), dict(lse=ODD4), dict(status=ODD4),
                dict(B=60000, N=30000, Hq=64, Hkv=64, max_pos=1 << 30)):
        assert chunk(lib, **bad) == binding.EINVAL, bad
    assert chunk(lib, nbytes=16) == binding.EWORKSPACE
    assert chunk(lib, ws=0x10080) == binding.EWORKSPACE
    need = binding_cache.spec_verify_attention_chunk_workspace_bytes
    assert need(2, 800, 32, 8, 128, 64) > 0 and need(1, 1 << 20, 64, 8, 64, 1 << 20) > 0
    for bad in ((0, 8, 32, 8, 128, 64), (2, 8, 32, 5, 128, 64), (2, 8, 32, 8, 130, 64), (2, 8, 32, 8, 128, 0)):
        assert need(*bad) == 0


def test_row_bytes(lib):
    for Hkv, D in ((1, 16), (8, 128), (3, 80), (5, 112), (16, 512)):
        assert binding_cache.spec_verify_kv_e4m3_row_bytes(Hkv, D) == pc.row_bytes(Hkv, D)
    for Hkv, D in ((0, 64), (1, 0), (1, 24), (1, 528), (1 << 20, 64)):
        assert binding_cache.spec_verify_kv_e4m3_row_bytes(Hkv, D) == 0


def test_tensors_on_the_host_are_refused(lib):
    h = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    c = torch.zeros((9, pc.row_bytes(2, 64)), dtype=torch.uint8)
    i = torch.zeros((1, 8), dtype=torch.int32)
    with pytest.raises(ValueError):
        binding_cache.spec_verify_kv_append_ex(h, h[:, :, :2], h[:, :, :2], c, c, i, i[0, :1], None)
    with pytest.raises(ValueError):
        binding_cache.spec_verify_kv_read(c, c, i, i[0, :1], 2, kv_heads=2, head_dim=64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding_cache.spec_verify_attention_e4m3(h, c, c, i, i[0, :1], kv_heads=2)
    with pytest.raises(ValueError):
        binding_cache.spec_verify_attention_chunk(h, c, c, i, i[0, :1], kv_heads=2)


def test_the_plain_form_of_the_rows():
    """What the GPU tests compare with: each of e4m3's values is its own nearest, and ties go to the even one."""
    g = pc.grid()[:127]
    x = torch.zeros((127, 1, 16), dtype=torch.float64)
    x[:, 0, 0], x[:, 0, 1] = g, 448.0
    rows = pc.encode(x, torch.bfloat16)
    assert torch.equal(rows[:, 0].long(), torch.arange(127)) and (rows[:, 16] == 127).all()
    assert torch.equal(pc.decode(rows, 1, 16), x)
    x[:126, 0, 0] = (g[1:] + g[:-1]) / 2
    rows = pc.encode(x, torch.bfloat16)[:126, 0].long()
    assert torch.equal(rows, torch.arange(126) + torch.arange(126) % 2)
    x = torch.tensor([1.0, 448.0, 448.1, 57344.0, 1e6, 2.0 ** -40]).double()[:, None, None].expand(6, 1, 16)
    assert (pc.encode(x, torch.float16)[:, 16].int() - 127).tolist() == [-8, 0, 1, 7, 7, -15]
    assert (pc.encode(x, torch.bfloat16)[:, 16].int() - 127).tolist() == [-8, 0, 1, 7, 7, -48]
