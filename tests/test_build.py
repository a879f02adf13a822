"""The build's files (CPU only, no compiler run): a build compiles into objects
of its own, links those, and leaves the libraries, the remarks and nothing else
behind; a failed one leaves what was there."""
import os
import subprocess

import pytest

from dense_bf16_gemm_amd import build


class Compiler:
    """Stands for hipcc: an output that names its inputs, a remark on stderr."""

    def __init__(self, fail=None):
        self.compiled, self.links, self.fail = [], [], fail

    def popen(self, cmd, stderr=None, **_):
        out, source = cmd[cmd.index("-o") + 1], os.path.basename(cmd[-1])
        self.compiled.append(out)
        with open(out, "w") as f:
            f.write(f"object of {source}\n")
        stderr.write(f"error in {source}\n" if source == self.fail else f"remark on {source}\n")

        class Done:
            returncode = 1 if source == self.fail else 0

            def wait(self):
                return self.returncode

        return Done()

    def run(self, cmd, check=False, **_):
        out = cmd[cmd.index("-o") + 1]
        objects = [a for a in cmd if a.endswith(".o")]
        self.links.append(objects)
        with open(out, "w") as f:
            for o in objects:
                f.write(open(o).read())


@pytest.fixture
def files(tmp_path, monkeypatch):
    for name, path in (("LIB", "libmm.so"), ("LIB_FULLSYNC", "libmm_fullsync.so"), ("BUILD_DIR", "_build"),
                       ("REMARKS", "_build/resource_usage.txt"),
                       ("REMARKS_DECODER", "_build/resource_usage_decoder.txt")):
        monkeypatch.setattr(build, name, str(tmp_path / path))

    def run(compiler):
        with monkeypatch.context() as m:
            m.setattr(subprocess, "Popen", compiler.popen)
            m.setattr(subprocess, "run", compiler.run)
            return build.build()

    return tmp_path, run


def test_two_builds_share_no_object(files):
    path, run = files
    first, second = Compiler(), Compiler()
    run(first)
    run(second)
    assert len(first.compiled) == len(set(first.compiled)) == 2 * len(build.SOURCES)
    assert not set(first.compiled) & set(second.compiled)
    for c in (first, second):
        assert sorted(o for objects in c.links for o in objects) == sorted(c.compiled)


def test_a_build_leaves_the_libraries_and_the_remarks(files):
    path, run = files
    run(Compiler())
    left = sorted(str(p.relative_to(path)) for p in path.rglob("*") if p.is_file())
    assert left == ["_build/resource_usage.txt", "_build/resource_usage_decoder.txt", "libmm.so", "libmm_fullsync.so"]
    for lib in ("libmm.so", "libmm_fullsync.so"):
        assert (path / lib).read_text() == "".join(f"object of {s}\n" for s in build.SOURCES)
    assert (path / "_build/resource_usage_decoder.txt").read_text() == "remark on mm_decoder.hip\n"


def test_a_failed_build_says_why_and_changes_nothing(files):
    path, run = files
    run(Compiler())
    before = {p: p.read_text() for p in path.rglob("*") if p.is_file()}
    with pytest.raises(RuntimeError, match="error in mm_decoder.hip"):
        run(Compiler(fail="mm_decoder.hip"))
    after = {p: p.read_text() for p in path.rglob("*") if p.is_file()}
    assert before == after
