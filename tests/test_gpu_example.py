"""The speculative-decoding example: what it decodes is what the model without a
cache chooses, token by token, up to choices that bf16 rounding leaves open."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from copy_reduce_dst_gb300 import _build  # noqa: E402

_build.build()
from copy_reduce_dst_gb300 import tb  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tree_decode_agrees_with_plain_greedy_decoding():
    spec = importlib.util.spec_from_file_location("tree_decode", os.path.join(ROOT, "examples", "tree_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model, texts, following = example.main(steps=6)
    assert texts[0][:21] == texts[1][:21] and max(len(t) for t in texts) > 21 + 6 + 4  # some drafts were accepted
    for text, after in zip(texts, following):
        logits = example.plain_logits(model, text)
        chosen = torch.tensor(text[21:] + [after], device="cuda")
        best, taken = logits[20:].max(-1).values, logits[20:].gather(1, chosen[:, None])[:, 0]
        # Both round activations to 16 bits about a dozen times a layer, by 2^-8 of
        # their size and not always the same way: sqrt(2 * 12) 2^-8 of the logits'
        # spread, twice (a difference), three deviations.  A wrong token is off by two.
        assert float((best - taken).max()) <= 0.12 * float(logits.std())


def test_readme_cache_example_runs():
    text = open(os.path.join(ROOT, "README.md")).read()
    code = text.split("```python")[2].split("```")[0]
    scope = {"torch": torch, "tb": tb}
    exec(compile(code, "README.md", "exec"), scope)
    torch.cuda.synchronize()
    assert scope["status"].tolist() == [0, 0, 0, 0]
    table, held, lens = scope["new"]
    assert lens.tolist() == [39, 39, 39, 0] and held.tolist() == [3, 3, 3, 0]
    assert table[1, :2].tolist() == table[0, :2].tolist() and int(table[1, 2]) != int(table[0, 2])
    assert scope["out"].isfinite().all()
