"""What the binding of include/msa_cache.h refuses before a call: tensors that do not live on the
current device, index caches of another shape or type than they are named (on stand-ins, as one
GPU or none is there)."""
import pytest
import torch


class Stub:
    """The part of a device tensor that the binding looks at."""

    def __init__(self, shape, dtype=torch.int32, device=0):
        self.shape, self.dtype, self.ndim = torch.Size(shape), dtype, len(shape)
        self.device = torch.device("cuda", device)
        self.is_cuda = True
        self.nbytes = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 0x10000

    def numel(self):
        return self.shape.numel()


@pytest.fixture
def B(monkeypatch):
    from block_sparse_paged_02_gb300 import binding
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)

    class Calls:  # nothing may be launched
        def __getattr__(self, name):
            return lambda *a: pytest.fail(f"{name} was called")

    monkeypatch.setattr(binding, "_calls", Calls)
    return binding


BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def batch(B, device=0, table=0):
    return B.make_batch(Stub((2,), device=device), Stub((2,), device=device), Stub((1,), device=device),
                        Stub((1, 4), device=table), 9, 2, max_q_len=2)


def attn(B, device=0, lse=0):
    kv = Stub((9, 128, 1, 128), BF, device)
    return B.make_attn_args(Stub((2, 8, 128), BF, device), kv, kv, B.MSA_KV_BF16, 9, Stub((2, 8, 128), BF, device),
                            Stub((2, 8), F32, lse), softmax_scale=0.1)


def pools(B, device=0, v=0, mass=0, index=0):
    kv = lambda d: Stub((9, 128, 1, 128), BF, d)
    return B.make_kv_pools(kv(device), kv(v), B.MSA_KV_BF16, mass=Stub((9, 128), F32, mass),
                           index=B.make_index_cache(kv(index), B.MSA_KV_BF16))


def test_structures_of_tensors_on_two_devices(B):
    for make in (lambda: batch(B, table=1), lambda: attn(B, lse=1), lambda: pools(B, v=1), lambda: pools(B, mass=1),
                 lambda: pools(B, index=1), lambda: B.make_cache_view(Stub((2,)), Stub((2, 4), device=1), 9),
                 lambda: B.make_tree(Stub((2, 1)), Stub((2, 4), device=1)),
                 lambda: B.make_index_cache(Stub((9, 128, 1, 64), U8), B.MSA_KV_FP8_E4M3, Stub((9, 128, 1), F32, 1))):
        with pytest.raises(ValueError, match="different devices"):
            make()


def test_calls_with_tensors_on_another_device(B):
    ws, st, mass = Stub((1 << 20,), U8), Stub((1,)), Stub((9, 128), F32)
    here = dict(b=batch(B), t=B.make_tree(Stub((2, 1))), a=attn(B), ws=ws, st=st, mass=mass)
    there = dict(b=batch(B, 1, 1), a=attn(B, 1, 1), ws=Stub((1 << 20,), U8, 1), st=Stub((1,), device=1),
                 mass=Stub((9, 128), F32, 1))
    trees = [B.make_tree(Stub((2, 1), device=1)), B.make_tree(None, Stub((2, 4), device=1))]
    for name, odd in [*there.items(), ("t", trees[0]), ("t", trees[1])]:
        x = {**here, name: odd}
        if name != "mass":
            with pytest.raises(ValueError, match="is current"):
                B.msa_tree_attn(x["b"], x["t"], x["a"], x["ws"], x["st"])
        with pytest.raises(ValueError, match="is current"):
            B.msa_attn_mass(x["b"], x["t"], x["a"], x["mass"], x["ws"], x["st"])
    view = lambda d=0: B.make_cache_view(Stub((2,), device=d), Stub((2, 4), device=d), 9)
    keep, kl = Stub((2, 8)), Stub((2,))
    for c, k, n in ((view(1), keep, kl), (view(), Stub((2, 8), device=1), kl), (view(), keep, Stub((2,), device=1))):
        with pytest.raises(ValueError, match="is current"):
            B.msa_evict_select(c, mass, 8, 0, 0, k, n, st)
        with pytest.raises(ValueError, match="is current"):
            B.msa_kv_compact(c, None, k, n, pools(B), st)
    with pytest.raises(ValueError, match="is current"):
        B.msa_kv_compact(view(), None, keep, kl, pools(B, 1, 1, 1, 1), st)


@pytest.mark.parametrize("dtype,tensor,scale", [
    (0, ((9, 128, 1, 64), U8), None),               # e4m3 codes named as bf16: rows of twice their bytes
    (1, ((9, 128, 1, 64), BF), None),
    (0, ((9, 64, 1, 128), BF), None),
    (1, ((9, 128, 1, 64), U8), ((9, 128), F32)),
    (1, ((9, 128, 2, 64), U8), ((9, 128, 1), F32)),  # a scale for one head of two
    (1, ((9, 128, 1, 64), U8), ((8, 128, 1), F32)),
    (1, ((9, 128, 1, 64), U8), ((9, 128, 1), BF))])
def test_index_cache_of_another_shape_or_type(B, dtype, tensor, scale):
    index = B.make_index_cache(Stub(*tensor), dtype, None if scale is None else Stub(*scale))
    kv = Stub((9, 128, 1, 128), BF)
    with pytest.raises(ValueError, match="index k_"):
        B.make_kv_pools(kv, kv, B.MSA_KV_BF16, index=index)


def test_index_caches_that_move(B):
    kv = Stub((9, 128, 1, 128), BF)
    for index in (B.make_index_cache(Stub((9, 128, 1, 128), BF), B.MSA_KV_BF16),
                  B.make_index_cache(Stub((9, 128, 2, 64), U8), B.MSA_KV_FP8_E4M3, Stub((9, 128, 2), F32)),
                  B.make_index_cache(Stub((9, 128, 1, 64), torch.float8_e4m3fn), B.MSA_KV_FP8_E4M3)):
        B.make_kv_pools(kv, kv, B.MSA_KV_BF16, index=index)
