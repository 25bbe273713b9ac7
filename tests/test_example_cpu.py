"""The example's function without a GPU."""
import importlib.util
import inspect
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_places_of_its_arguments():
    """A call by position means what it meant before dropout joined: that comes last."""
    spec = importlib.util.spec_from_file_location(
        "embedding_classifier", os.path.join(ROOT, "examples", "embedding_classifier.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert list(inspect.signature(m.train).parameters) == [
        "steps", "rows", "dim", "classes", "bags", "bag", "seed", "log", "dropout"]
