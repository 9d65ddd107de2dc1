"""The layers refuse what their calls would misread: fewer offsets than the
experts need, before any kernel could read past them, and tokens of another form."""
import pytest
import torch


def layers():
    from tiled_layout_algebra_amd.expert_layer import ExpertLayer
    from tiled_layout_algebra_amd.gated_layer import GatedLayer
    t = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16)  # noqa: E731
    for experts in (1, 3):
        e = ExpertLayer(t(experts, 8, 16), t(experts, 16), t(experts, 16, 8))
        g = GatedLayer(t(experts, 32, 8), t(experts, 8, 16))
        for call in (e.forward, e.decode, g.forward, g.serve):
            yield experts, call


def test_too_few_offsets():
    x = torch.zeros(5, 8, dtype=torch.bfloat16)
    for experts, call in layers():
        for n in range(experts + 1):
            with pytest.raises(ValueError, match="offsets must hold %d values" % (experts + 1)):
                call(x, torch.zeros(n, dtype=torch.int32))


def test_tokens_that_would_be_misread():
    from tiled_layout_algebra_amd.gated_layer import quantize_tokens
    for x in (torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.float16),
              torch.zeros(4, 16, dtype=torch.bfloat16)[:, ::2], torch.zeros(8, 4, dtype=torch.bfloat16).t()):
        with pytest.raises(ValueError, match="x must be a contiguous bfloat16"):
            quantize_tokens(x)
