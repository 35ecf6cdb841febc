"""Sizes beyond the C entry points' int32 are refused by the binding: cut to 32 bits they would be other sizes, and a
part of the rows would be left as it was without a word."""
import pytest
import torch

BIG = (1 << 32) + 4  # 4, cut to 32 bits


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_ffn_rms_gb300 as M
    return M


def rows(n, h, dtype=torch.bfloat16):
    return torch.zeros((1, 1), dtype=dtype).expand(n, h)


def test_sizes_beyond_int32(M):
    f32 = torch.float32
    big, w, few = rows(BIG, 8), torch.ones(8, dtype=torch.bfloat16), rows(4, 8)
    row, vec = rows(1, BIG, torch.int32)[0], rows(1, BIG, f32)[0]
    wide = rows(4, (1 << 32) + 8)
    ws = torch.zeros(1024, dtype=torch.uint8)
    f8 = torch.zeros(8)
    calls = [
        lambda: M.moe_unpermute(big, row, big, BIG, 1),
        lambda: M.moe_unpermute(few, torch.zeros(4, dtype=torch.int32), few, 4, (1 << 32) + 1),
        lambda: M.moe_unpermute(wide, torch.zeros(4, dtype=torch.int32), wide, 4, 1),
        lambda: M.moe_permute_backward(big, row, big, BIG, 1),
        lambda: M.moe_unpermute_backward(big, big, row, rows(BIG, 1, f32), BIG, 1, dy=big),
        lambda: M.moe_unpermute_backward(few, few, row[:4], rows(4, 1, f32), 4, 1, ids=rows(4, 1, torch.int32),
                                         dlogits=rows(4, BIG, f32)),
        lambda: M.moe_layernorm(big, w, 1e-6, big),
        lambda: M.moe_layernorm(wide, rows(1, (1 << 32) + 8)[0], 1e-6, wide),
        lambda: M.moe_layernorm_backward(big, big, w, vec, vec, big, f8, ws),
        lambda: M.moe_rmsnorm_backward(big, big, w, 1e-6, big, f8, ws),
        lambda: M.moe_linear(big, few, rows(BIG, 4)),
        lambda: M.moe_linear(few, big, rows(4, BIG)),
        lambda: M.moe_linear(few, few, rows(4, 4), act=1 << 32),
        lambda: M.moe_linear_backward(rows(BIG, 4), big, few, ws, db=f8),
        lambda: M.moe_linear_backward(rows(4, BIG), few, big, ws, dx=few),
        lambda: M.moe_norm_backward_workspace_size(BIG, 8),
        lambda: M.moe_norm_backward_workspace_size(4, (1 << 32) + 8),
        lambda: M.moe_linear_backward_workspace_size(BIG, 8, 8),
        lambda: M.moe_linear_backward_workspace_size(4, (1 << 32) + 8, 8),
        lambda: M.moe_linear_backward_workspace_size(4, 8, (1 << 32) + 8),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="int32"):
            call()
            pytest.fail(f"call {i} went through")


def test_negative_sizes_keep_their_error(M):
    with pytest.raises(M.MoeError):
        M.moe_norm_backward_workspace_size(-1, 8)
    with pytest.raises(M.MoeError):
        M.moe_linear_backward_workspace_size(-1, 8, 8)
