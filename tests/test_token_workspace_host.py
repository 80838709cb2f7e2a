"""Workspaces that do not hold the bytes they seem to, before any device work (CPU)."""

import pytest

torch = pytest.importorskip("torch")

from io_aware_exact_30_b200 import attn  # noqa: E402


def test_a_workspace_repeated_in_place_is_refused():
    """An expanded tensor counts elements that it does not own: the kernels would write
    past its memory."""
    B, H, N, d = 1, 1, 2000, 64
    need = attn.attn_decay_workspace_bytes(B, H, N, d)
    back = attn.attn_decay_workspace_bytes(B, H, N, d, True)
    split = attn.attn_cache_attend_workspace_bytes(B, H, H, 1, d, 4096)
    assert need > 0 and back > 0 and split > 0
    x = torch.zeros(B, H, N, d, dtype=torch.bfloat16)
    ld = torch.zeros(H)
    for ws in (torch.zeros(16, dtype=torch.uint8).expand(1 << 22, 16), torch.zeros(1).expand(1 << 22),
               torch.zeros(1 << 22, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            attn.attn_decay_fwd(x, x, x, ld, x, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            attn.attn_decay_bwd(x, x, x, ld, x, x, x, x, workspace=ws)
        q = x[:, :, :1].contiguous()
        codes = torch.zeros(64, H, 64, d, dtype=torch.uint8)
        cache = attn.Cache8(codes, codes.clone(), torch.zeros(64, H), torch.zeros(64, H))
        with pytest.raises(ValueError, match="workspace"):
            attn.attn_cache_attend(q, cache, torch.zeros(B, 64, dtype=torch.int32), torch.zeros(B, dtype=torch.int32),
                                   q.clone(), torch.zeros(B, H, 1), ws)
