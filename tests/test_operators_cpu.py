"""Host-side refusals of the operators around verification (KV append, attention, log probabilities):
every call below fails its checks before anything is launched, so no GPU is needed."""
import ctypes

import pytest
import torch

from speculative_decoding_verification_verify_gb300 import _build, binding

P = ctypes.c_void_p
A, ODD, ODD4 = 0x10000, 0x10008, 0x10002  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load_library()


def append(lib, **bad):
    a = dict(q=A, k=A, v=A, dtype=0, qs=48 * 128, ks=48 * 128, vs=48 * 128, q_out=A, kc=A, vc=A, slots=100, kss=1024,
             vss=1024, table=A, max_pos=64, committed=A, parents=None, num_nodes=None, cs=A, positions=64, rot=128,
             interleaved=0, B=2, N=8, Hq=32, Hkv=8, D=128, status=None, stream=None)
    assert set(bad) <= set(a)
    return lib.spec_verify_kv_append(*{**a, **bad}.values())


def test_append(lib):
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(q_out=None), dict(kc=None), dict(vc=None),
                dict(table=None), dict(committed=None), dict(dtype=1), dict(dtype=7), dict(B=0), dict(N=0),
                dict(parents=A, N=65), dict(max_pos=0), dict(slots=0), dict(slots=1 << 31), dict(Hq=0), dict(Hkv=0),
                dict(D=120), dict(D=8), dict(D=2048), dict(rot=8), dict(rot=144), dict(rot=-16), dict(cs=None),
                dict(positions=0), dict(qs=32 * 128 - 8), dict(qs=48 * 128 + 4), dict(ks=1016), dict(vs=1016),
                dict(kss=1016), dict(vss=1020), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(q_out=ODD), dict(kc=ODD),
                dict(vc=ODD), dict(cs=ODD), dict(table=ODD4), dict(committed=ODD4), dict(parents=ODD4),
                dict(num_nodes=ODD4), dict(status=ODD4), dict(B=1 << 16, N=1 << 16)):
        assert append(lib, **bad) == binding.EINVAL, bad


def attention(lib, **bad):
    a = dict(q=A, dtype=0, qs=32 * 128, kc=A, vc=A, slots=100, kss=1024, vss=1024, table=A, max_pos=64, committed=A,
             parents=None, num_nodes=None, B=2, N=8, Hq=32, Hkv=8, D=128, scale=0.1, out=A, lse=None, ws=A,
             nbytes=1 << 30, status=None, stream=None)
    assert set(bad) <= set(a)
    return lib.spec_verify_attention(*{**a, **bad}.values())


def test_attention(lib):
    for bad in (dict(q=None), dict(kc=None), dict(vc=None), dict(table=None), dict(committed=None), dict(out=None),
                dict(ws=None), dict(dtype=1), dict(B=0), dict(B=65537), dict(N=0), dict(N=65), dict(Hq=0), dict(Hkv=0),
                dict(Hkv=5), dict(D=48), dict(D=72), dict(D=144), dict(max_pos=0), dict(slots=0), dict(slots=1 << 31),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(qs=4088),
                dict(qs=4100), dict(kss=1016), dict(vss=1028), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD),
                dict(table=ODD4), dict(committed=ODD4), dict(parents=ODD4), dict(num_nodes=ODD4), dict(lse=ODD4),
                dict(status=ODD4)):
        assert attention(lib, **bad) == binding.EINVAL, bad
    assert attention(lib, nbytes=16) == binding.EWORKSPACE
    assert attention(lib, ws=0x10080) == binding.EWORKSPACE
    need = binding.spec_verify_attention_workspace_bytes
    assert need(2, 8, 32, 8, 128, 64) > 0 and need(65536, 64, 64, 1, 64, 1 << 20) > 0
    for bad in ((0, 8, 32, 8, 128, 64), (2, 65, 32, 8, 128, 64), (2, 8, 32, 5, 128, 64), (2, 8, 32, 8, 130, 64),
                (2, 8, 32, 8, 128, 0)):
        assert need(*bad) == 0


def logprobs(lib, **bad):
    a = dict(logits=A, dtype=0, tokens=A, index=None, B=2, rows=8, T=8, V=1000, temps=None, temp=1.0, top=5, lp=A, ent=A,
             ranks=A, ids=A, tlp=A, ws=A, nbytes=1 << 30, status=None, stream=None)
    assert set(bad) <= set(a)
    return lib.spec_verify_logprobs(*{**a, **bad}.values())


def test_logprobs(lib):
    for bad in (dict(logits=None), dict(tokens=None), dict(lp=None), dict(ws=None), dict(dtype=2), dict(dtype=-1),
                dict(B=0), dict(B=65537), dict(rows=0), dict(rows=65), dict(T=0), dict(T=65), dict(T=9), dict(V=0),
                dict(top=33), dict(top=-1), dict(ids=None), dict(tlp=None), dict(temp=-0.5), dict(temp=float("nan")),
                dict(temp=float("inf")), dict(logits=0x10001), dict(dtype=1, logits=0x10002), dict(tokens=ODD4),
                dict(index=ODD4), dict(temps=ODD4), dict(lp=ODD4), dict(ent=ODD4), dict(ranks=ODD4), dict(ids=ODD4),
                dict(tlp=ODD4), dict(status=ODD4)):
        assert logprobs(lib, **bad) == binding.EINVAL, bad
    assert logprobs(lib, nbytes=16) == binding.EWORKSPACE
    assert logprobs(lib, ws=0x10010) == binding.EWORKSPACE
    need = binding.spec_verify_logprobs_workspace_bytes
    assert need(2, 8, 1000, 5) > 0 and need(65536, 64, 1 << 30, 32) > 0
    for bad in ((0, 8, 1000, 5), (2, 65, 1000, 5), (2, 8, 0, 5), (2, 8, 1000, 33)):
        assert need(*bad) == 0


def test_tensors_on_the_host_are_refused(lib):
    h = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    c = torch.zeros((9, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 8), dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.spec_verify_kv_append(h, h[:, :, :2], h[:, :, :2], c, c, i, i[0, :1], None)
    with pytest.raises(ValueError):
        binding.spec_verify_attention(h, c, c, i, i[0, :1])
    with pytest.raises(ValueError):
        binding.spec_verify_logprobs(torch.zeros((1, 2, 9)), i[:, :2])
