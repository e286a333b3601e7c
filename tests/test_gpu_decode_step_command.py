"""latency_collectives_amd.decode_step as a command: what its texts say that it runs, it runs."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture
def calls(monkeypatch):
    """The names of the package's calls, in order."""
    import latency_collectives_amd as lc
    from latency_collectives_amd import decode_step

    seen = []

    class Spy:
        def __getattr__(self, name):
            inner = getattr(lc, name)
            if not callable(inner):
                return inner

            def call(*a, **k):
                seen.append(name)
                return inner(*a, **k)

            return call

    monkeypatch.setattr(decode_step, "lc", Spy())
    return seen


def run(*extra):
    from latency_collectives_amd import decode_step

    decode_step.main(["--ranks", "2", "--layers", "1", "--requests", "5", "--prompt", "70", "--steps", "3", *extra])
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", ["4", "8"])
def test_samples_are_forked_freed_and_moved_together(calls, bits):
    run("--bits", bits, "--samples", "3")
    pages = [n for n in calls if n.startswith("ar_pages_") and n != "ar_pages_scratch"]
    assert pages == ["ar_pages_fork", "ar_pages_copy", "ar_pages_free", "ar_pages_compact", "ar_pages_copy", "ar_pages_free"]
    # a step after the pages have moved
    assert f"ar_kv{bits}_attention" in calls[calls.index("ar_pages_compact"):]


def test_only_packed_prompts_take_their_workspace(calls):
    run("--bits", "8")
    assert "ar_prompt_create" not in calls and "ar_prompt_destroy" not in calls
    run("--bits", "8", "--packed")
    assert calls.count("ar_prompt_create") == calls.count("ar_prompt_destroy") == 1


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
def test_workspaces_have_the_sizes_that_the_header_gives(d):
    """69 to 102 MB, in whole steps of the allocator's 2 MiB."""
    import latency_collectives_amd as lc

    for make, end in ((lambda: lc.ar_kv8_create(2, d, 16), lc.ar_kv8_destroy), (lambda: lc.ar_prompt_create(2, d), lc.ar_prompt_destroy)):
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        h = make()
        took = before - torch.cuda.mem_get_info()[0]
        end(h)
        assert 69e6 - 1 <= took <= 102.5e6 + 2 * 2 ** 20, took


def test_prompts_without_steps(capsys):
    run("--steps", "0")
    assert "us a decode step" in capsys.readouterr().out
