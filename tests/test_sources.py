"""What the CUDA sources may not hold, read as text (no GPU needed)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "combine_route_count_prefix_gb300", "**", "*.cu*"), recursive=True))


def bulk_copies(text):
    """The mnemonics of the bulk copies in a source's inline PTX, string pieces joined."""
    text = re.sub(r'"\s*"', "", text)
    return re.findall(r"cp\.async\.bulk[a-zA-Z0-9_.:]*", text)


def test_bulk_copies_are_found():
    assert bulk_copies('asm("cp.async.bulk.tensor.2d.shared::cluster"\n   ".global.multicast::cluster [%0]")') == [
        "cp.async.bulk.tensor.2d.shared::cluster.global.multicast::cluster"]
    assert sum(len(bulk_copies(open(f).read())) for f in SOURCES) > 4


def test_no_load_is_multicast_to_a_cluster():
    """The library serves jobs of several GPUs, and its tensor maps cover
    whatever address a caller gives: a multicast load of another GPU's memory
    must not be possible, so every CTA fetches what it needs itself."""
    for f in SOURCES:
        for copy in bulk_copies(open(f).read()):
            assert "multicast" not in copy, (os.path.basename(f), copy)
