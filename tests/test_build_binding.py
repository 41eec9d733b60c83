"""The compiled half of the block operators' binding is a module of one Python:
its file carries that Python's tag, so that another one on the same tree builds
its own instead of loading this one."""
import os
import sysconfig

from transformer_layer_non_gb300 import build as lsbuild


def test_the_file_names_its_python():
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert suffix.count(".") == 2  # a tag and .so
    assert os.path.basename(lsbuild.BINDING_LIB) == "_ls_block_call" + suffix


def test_it_is_built_there():
    path = lsbuild.build_binding()
    assert path is None or (path == lsbuild.BINDING_LIB and os.path.exists(path))
