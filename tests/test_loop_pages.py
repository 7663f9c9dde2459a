"""runtime.AttentionLoop refuses tokens that its pages cannot hold when it is made, not in a step (whose
scheduler has admitted requests by then)."""

from types import SimpleNamespace

import pytest

from heterogeneous_lora_amd import runtime as rt


class Reached(Exception):
    pass


def pages_taken(monkeypatch, page_elems, heads, dim, **kw):
    """Tokens to a page of a loop that gets as far as taking a GPU's memory."""
    def stop(self, *args, **options):
        raise Reached(options["tokens_per_page"])
    monkeypatch.setattr(rt.ServingLoop, "__init__", stop)
    with pytest.raises(Reached) as e:
        rt.AttentionLoop(SimpleNamespace(page_elems=page_elems), 10, 2 * heads, heads, dim, 100, **kw)
    return e.value.args[0]


def refused(match, page_elems, heads, dim, **kw):
    with pytest.raises(ValueError, match=match):
        rt.AttentionLoop(SimpleNamespace(page_elems=page_elems), 10, 2 * heads, heads, dim, 100, **kw)


# (a token of 4 heads of 128 in 4 bits: 272 bytes, in 16: 1024)
@pytest.mark.parametrize("page_elems,kw,pages", [(512, dict(), 1), (1024, dict(tokens_per_page=2), 2), (512, dict(kv_bits=4), 3),
                                                 (136, dict(kv_bits=4), 1), (512, dict(kv_bits=4, tokens_per_page=2), 2)])
def test_taken(monkeypatch, page_elems, kw, pages):
    assert pages_taken(monkeypatch, page_elems, 4, 128, **kw) == pages


@pytest.mark.parametrize("page_elems,kw", [(504, dict()), (512, dict(tokens_per_page=2)), (128, dict(kv_bits=4)),
                                           (512, dict(kv_bits=4, tokens_per_page=4))])
def test_refused(page_elems, kw):
    refused("do not fit a page", page_elems, 4, 128, **kw)


def test_refused_bits():
    refused("kv_bits", 512, 4, 128, kv_bits=8)
