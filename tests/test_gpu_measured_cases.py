"""The measured cases' calls of libgk under a stream that is not the default one: each state's context is its stream's."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["attn_one_token", "store_decode", "read_one", "sample_one", "w4_one"])
def test_cases_under_a_side_stream(monkeypatch, name):
    import torch

    from perf import operators

    monkeypatch.setattr(operators, "own", True)
    case = next(c for c in operators.listed() if c["name"] == name)

    def outputs():
        out = operators.run(operators.prepare(case, 3))
        return [x.clone() for x in (out if isinstance(out, tuple) else (out,))]

    want = outputs()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # the stream is about 10 ms behind the host: nothing is there yet by chance
        context = operators.prepare(case, 3)["ctx"]
        got = outputs()
        assert operators.prepare(case, 3)["ctx"] is context
    assert operators.prepare(case, 3)["ctx"] is not context
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
