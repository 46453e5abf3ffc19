"""The example decoder layer: append, attention, router and experts together."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import kv_cache as K  # noqa: E402


def _check(layer, seqs, q, out, n_q):
    """The layer's attention against float64 over the entries its cache holds."""
    at = 0
    for b, m in enumerate(n_q):
        n = int(seqs.lens[b])
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        k, v = (t.double().cpu().numpy() for t in layer.kv.gather(
            seqs.place(torch.full((n,), b, device="cuda"), pos), out_dtype=torch.float32))
        ref = K.attention(q[at:at + m].double().cpu().numpy(), k, v, layer.head_dim ** -0.5)
        assert K.check_attention(out[at:at + m].float().cpu().numpy(), None, ref, n, np.abs(v).max()) == (0, 0)
        at += m


def test_prompts_then_tokens_attend_to_what_was_appended():
    from examples.decoder_layer import DecoderLayer, Sequences
    layer, seqs = DecoderLayer(), Sequences(3, 256)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for n_q in ([70, 1, 140], [3, 20, 0], [1, 1, 1]):
        x = torch.randn(sum(n_q), 512, generator=gen, device="cuda", dtype=torch.bfloat16)
        b = seqs.prompts(n_q) if n_q != [1, 1, 1] else seqs.step()
        _check(layer, seqs, *layer.attention(x, b), n_q)
    assert layer.kv.status() == 0


def test_steps_from_a_graph_equal_steps_called_one_by_one():
    from examples.decoder_layer import DecoderLayer, Sequences, main
    n_q = (90, 5, 64)
    torch.manual_seed(3)
    _, seqs, rows = main(n_q, steps=4)
    torch.manual_seed(3)
    layer, again = DecoderLayer(), Sequences(3, 512)
    x = torch.randn(sum(n_q), 512, device="cuda", dtype=torch.bfloat16)
    y = layer(x, again.prompts(list(n_q)))[torch.tensor(n_q).cumsum(0).cuda() - 1]
    for _ in range(4):
        y = layer(y, again.step())
    assert torch.equal(seqs.lens, again.lens)
    assert torch.equal(y, rows) and bool(torch.isfinite(y.float()).all())
