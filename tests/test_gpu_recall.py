"""The example that trains and serves a small model."""
import pytest
import torch

from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu


def test_the_model_learns_and_serves():
    from examples import recall

    torch.manual_seed(0)
    model = recall.Recall().cuda()
    losses = recall.train(model, 120)
    assert losses[-1] < 0.5 * losses[0]
    prompts = [[3, 9, 1, 3], [5], [60, 2, 33, 21, 8, 60, 2]]
    u = torch.rand((6, 3), generator=torch.Generator().manual_seed(2)).cuda()
    written, state = recall.serve(model, prompts, 6, u, top_k=10, top_p=0.9)
    assert written.shape == (6, 3) and bool(((written >= 0) & (written < model.vocab)).all())
    # The states that the steps left are the definition's over all tokens.
    host = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
    for r, prompt in enumerate(prompts):
        tokens = torch.tensor(prompt + written[:, r].tolist()).cuda()
        before = torch.cat([torch.tensor([model.vocab]).cuda(), tokens[:-1]])
        q, k, v = (host(t) for t in model.rows(tokens, before))
        g = model.log_decay.cpu().numpy()
        want = ref.forward(q, k, v, g, model.scale, [len(tokens)])[1][0]
        size = ref.forward(abs(q), abs(k), abs(v), g, model.scale, [len(tokens)])[1][0]
        off = abs(host(state[r]) - want)
        # 32-bit sums and powers over the tokens, and the rows' own products,
        # whose sums over 128 may differ by their order before a bf16 rounding.
        assert (off <= (len(tokens) + 128) * 2.0 ** -23 * size + 4 * 2.0 ** -8 * size).all()
