"""The serving operators' dispatcher entries without a GPU: shapes and types of
the fake implementations, and what they refuse."""
import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")
import epilogue_scaled_gemm_amd.torch_ops  # noqa: E402,F401

ops = torch.ops.lingemm
BF16 = torch.bfloat16


def meta(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_fake_shapes():
    q, k = meta(7, 8, 64), meta(7, 2, 64)
    a, b = ops.qk_norm_rope(q, k)
    assert a.shape == q.shape and b.shape == k.shape and a.dtype == BF16
    cache = meta(4, 2, 16, 64)
    i = meta(7, dtype=torch.int32)
    assert ops.kv_append(k, k, cache, cache.clone(), i).shape == (0,)
    assert ops.kv_append(k, k, cache, cache.clone(), i, q=q).shape == q.shape
    out, lse = ops.tree_attention(q, cache, cache, meta(2, 3, dtype=torch.int32),
                                  meta(2, dtype=torch.int32), meta(3, dtype=torch.int32), 40, 4)
    assert out.shape == q.shape and out.dtype == BF16
    assert lse.shape == (7, 8) and lse.dtype == torch.float32
    lp, en, ids, best = ops.token_logprobs(meta(7, 1000), i, top=5)
    assert lp.shape == en.shape == (7,) and lp.dtype == torch.float32
    assert ids.shape == best.shape == (7, 5) and ids.dtype == torch.int32


def test_fakes_refuse():
    with pytest.raises(ValueError):
        ops.qk_norm_rope(meta(7, 8, 64, dtype=torch.float32), meta(7, 2, 64))
    with pytest.raises(ValueError):
        ops.qk_norm_rope(meta(7, 512), meta(7, 2, 64))
    with pytest.raises(ValueError):
        ops.token_logprobs(meta(1000), meta(1, dtype=torch.int32))


def test_cpu_tensors_are_refused():
    q = torch.zeros(2, 2, 64, dtype=BF16)
    with pytest.raises(Exception):
        ops.qk_norm_rope(q, q)


def test_the_cache_is_marked_as_written():
    schema = ops.kv_append.default._schema
    written = {a.name for a in schema.arguments if a.alias_info is not None and a.alias_info.is_write}
    assert written == {"k_cache", "v_cache"}
