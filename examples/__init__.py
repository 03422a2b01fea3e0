"""Programs that use the framework."""
