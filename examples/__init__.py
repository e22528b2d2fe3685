"""Programs that use the library's entry points together."""
