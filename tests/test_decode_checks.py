"""What the binding and the examples check on the host before a call of the cache, the attention and the
verification, without a GPU."""

import pytest
import torch

import weight_streaming_linear_amd as wsl

CPU = torch.device("cpu")


@pytest.mark.parametrize("shape", [(2, 3, 7), (1, 3, 7), (4, 1, 7), (2, 2, 1)])
@pytest.mark.parametrize("step", [0, 1])
def test_rows_that_lie_over_each_other_are_no_rows(shape, step):
    """Broadcast rows (a drafter with one distribution for every position), and rows that overlap: a step
    below vocab from row to row must not be handed on, least of all 0, which could stand for no rows."""
    n, rows, vocab = shape
    wide = torch.zeros(n * rows + vocab)
    t = wide.as_strided(shape, (rows * step, step, 1))
    if step >= vocab:
        assert wsl._prob_rows(t, "q", CPU, shape) == vocab
        return
    with pytest.raises(ValueError, match="q: rows"):
        wsl._prob_rows(t, "q", CPU, shape)


def test_rows_of_their_own_keep_their_step():
    wide = torch.zeros(2, 3, 11)
    assert wsl._prob_rows(wide, "p", CPU, (2, 3, 11)) == 11
    assert wsl._prob_rows(wide[..., 2:9], "p", CPU, (2, 3, 7)) == 11
    assert wsl._prob_rows(wide[:, :1, :7], "p", CPU, (2, 1, 7)) == 33
    assert wsl._prob_rows(wide[:1, 1:2, :7], "p", CPU, (1, 1, 7)) == 7
    assert wsl._prob_rows(wide[:0], "p", CPU, (0, 3, 11)) == 11


def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class _Model:
    """What decode() asks a model before it runs it; running it is a mistake of its own here."""

    class Ran(Exception):
        pass

    def __init__(self, pages, page=16):
        self.table, self.page = torch.zeros((2, pages), dtype=torch.int32), page

    def step(self, tokens, lens):
        raise self.Ran


@pytest.mark.parametrize("pages,fits", [((7, 7), True), ((6, 7), False), ((7, 6), False), ((1, 1), False)])
def test_the_example_counts_its_tokens_before_it_starts(pages, fits):
    """70 tokens and 8 rounds of 4 drafts and a token: 110, all of which may stand."""
    ex = _example()
    models = [_Model(n) for n in pages]
    prompt = torch.zeros((2, 70), dtype=torch.int32)
    with pytest.raises(_Model.Ran if fits else ValueError):
        ex.decode(*models, prompt, 4, 8, lambda n, m: torch.zeros(n, m))


def test_the_example_makes_room_for_what_it_is_asked_for(monkeypatch):
    ex = _example()
    made = []

    class Decoder(_Model):
        vocab = 8000

        def __init__(self, n_seq, layers, capacity=1024, page=16, **kw):
            super().__init__(-(-capacity // page), page)
            made.append(self)

    monkeypatch.setattr(ex, "Decoder", Decoder)
    for name in ("randint", "zeros"):
        plain = getattr(torch, name)
        monkeypatch.setattr(ex.torch, name, lambda *a, device=None, plain=plain, **kw: plain(*a, **kw))
    generator = torch.Generator
    monkeypatch.setattr(ex.torch, "Generator", lambda device=None: generator())
    monkeypatch.setattr("sys.argv", ["speculative_decode.py", "--tokens", "5000", "--width", "7"])
    with pytest.raises(_Model.Ran):         # past the check, into the first step
        ex.main()
    assert made and all(m.table.shape[1] * m.page >= 100 + 5000 for m in made)


def test_the_division_of_the_attention_work(tmp_path):
    """attn_plan on 64 simulated lanes, unset variables filled with a pattern."""
    import os
    import shutil
    import subprocess
    here = os.path.dirname(os.path.abspath(__file__))
    clang = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "clang++")
    clang = clang if os.path.exists(clang) else shutil.which("clang++")
    if clang is None:
        pytest.skip("clang++ not available")
    exe = str(tmp_path / "attn_plan")
    subprocess.run([clang, "-std=c++17", "-O1", "-ftrivial-auto-var-init=pattern", "-isystem", os.path.join(here, "cpp", "wave"),
                    os.path.join(here, "cpp", "attn_plan_main.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr


def test_contiguous_tensors_still_need_a_unit_last_step():
    """As from the first: a contiguous tensor whose last dimension has one entry and another step is refused."""
    from types import SimpleNamespace

    def like(t):
        return SimpleNamespace(is_cuda=True, dtype=t.dtype, device=t.device, dim=t.dim, numel=t.numel, stride=t.stride,
                               is_contiguous=t.is_contiguous)

    odd = torch.zeros(64).as_strided((5, 1), (1, 7))
    assert odd.is_contiguous()
    for contiguous in (False, True):
        with pytest.raises(ValueError, match="last dimension"):
            wsl._require(like(odd), "y", (torch.float32,), contiguous=contiguous)
        wsl._require(like(torch.zeros(5, 1)), "y", (torch.float32,), contiguous=contiguous)
