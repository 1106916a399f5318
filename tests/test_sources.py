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


def function_bodies(text, head):
    """The bodies of the functions whose text before the brace matches `head`."""
    for m in re.finditer(head, text):
        start = at = text.index("{", m.end())
        depth = 0
        while True:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
            if depth == 0:
                break
        yield text[start:at]


def test_row_scales_of_kernels_that_start_early_are_not_read_as_constants():
    """A kernel that starts before the one that writes its rows' scales has ended may not
    read them with __ldg, which is for what nobody writes while the kernel runs."""
    def read(name):
        return open(os.path.join(ROOT, "combine_route_count_prefix_gb300", "csrc", name)).read()

    early = [b for name, head in (("gemm_int8.cu", r"\nk_int8_few\("), ("gemm_int8_tiles.cu", r"\nk_int8_tiles\("),
                                  ("few_tokens.cu", r"\nk_few_gate_up\("), ("few_tokens.cu", r"\nk_few_down\("),
                                  ("gemm_small.cu", r"else if \(EPI == \(int\)Epi::Linear\)"),
                                  ("gemm_tc.cu", r"else if \(EPI == \(int\)Epi::Linear\)"))
             for b in function_bodies(read(name), head)]
    assert len(early) == 6
    for body in early:
        assert re.search(r"\b(qs|s2|row_scales)\b", body)
        assert not re.search(r"__ldg\([^;]*\b(p\.qs|p\.s2|row_scales|s2)\b", body)


def test_nothing_in_the_sources_is_without_a_user():
    """Device functions, constants and macros that only their definition names."""
    text = re.sub(r"//[^\n]*", "", "\n".join(open(f).read() for f in SOURCES))
    names = set()
    for pattern in (r"__device__\s+(?:__forceinline__|__noinline__|inline)\s+[\w:<> ]+?[\s&*](\w+)\s*\(",
                    r"constexpr\s+[\w:<> ]+?\s(\w+)\s*[=({]", r"#define\s+(\w+)"):
        names.update(re.findall(pattern, text))
    assert len(names) > 200
    assert [n for n in sorted(names - {"operator"}) if len(re.findall(rf"\b{n}\b", text)) < 2] == []
