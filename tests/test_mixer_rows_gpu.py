"""The Mamba-2 mixer's operators on the GPU where tests/test_mixer_gpu.py does not
reach: prompts cut into segments beside other work on the card.  Problems,
references and bounds as there."""
import pytest

from test_mixer_gpu import Mix, dev, ssm  # noqa: F401  (fixtures)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_cut_prompts_beside_other_work(ssm, dev):  # noqa: F811
    """Prompts of four segments that continue from their slots, with products on
    another stream holding parts of the card: the last segment of a sequence
    may end before its first one starts, and writes the slot that the sequence
    started from.  Every call gives the quiet call's bits."""
    def fresh():
        return Mix(dev, (256, 200), 24, 64, 1, 128, 4, "bf16", 1000, gate=False, has=True)
    quiet = fresh()
    quiet.run(ssm)
    torch.cuda.synchronize()
    quiet.check("quiet")
    m = fresh()
    keep = m.cs.clone(), m.hs.clone()
    a = torch.randn(4096, 4096, device=dev).bfloat16()
    out = torch.empty_like(a)
    side = torch.cuda.Stream(dev)
    for _ in range(20):
        m.cs.copy_(keep[0]), m.hs.copy_(keep[1])
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            for _ in range(3):
                torch.mm(a, a, out=out)
        m.run(ssm)
        torch.cuda.synchronize()
        assert torch.equal(m.y, quiet.y) and torch.equal(m.hs, quiet.hs) and torch.equal(m.cs, quiet.cs)
